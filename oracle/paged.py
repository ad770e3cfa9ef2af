"""Oracle of the paged 4-bit KV cache in numpy fp64: the quantiser, the pool's
byte format and ragged attention with a window and sinks, written out token by
token from the definitions in include/sf.h (sf_kvp).  It shares no code with
the CUDA path.

The abstract's low-bit KV caches are the source of the 4-bit format ("StrataFlux:
Memory-Hierarchy-Native Low-Bit LLM Inference"); pages, ragged queries, windows
and sinks are the usual definitions.
"""
from __future__ import annotations

import numpy as np

LIMIT = 65408.0


def quantise(x):
    """x [..][d] float64 -> codes [..][d] uint8, s and m [..][d/32] float16."""
    x = np.asarray(x, np.float64)
    w = np.clip(np.where(np.isnan(x), 0.0, x), -LIMIT, LIMIT).reshape(*x.shape[:-1], -1, 32)
    lo, hi = w.min(-1), w.max(-1)
    s, m = ((hi - lo) / 15.0).astype(np.float16), lo.astype(np.float16)
    sd, md = s.astype(np.float64)[..., None], m.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.floor((w - md) / sd + 0.5)
    q = np.where(sd == 0.0, 0.0, np.clip(q, 0.0, 15.0))
    return q.astype(np.uint8).reshape(x.shape), s, m


def values(codes, s, m):
    """The fp64 values m + s q."""
    g = codes.reshape(*codes.shape[:-1], -1, 32).astype(np.float64)
    return (m.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * g).reshape(codes.shape)


def stored(x):
    return values(*quantise(x))


class Pool:
    """The bytes of a pool, written and read one token at a time."""

    def __init__(self, n_pages, page, h_kv, d, fill=0):
        self.n_pages, self.page, self.h_kv, self.d = n_pages, page, h_kv, d
        self.tile_bytes = 20 * d
        self.bytes = np.full(n_pages * h_kv * (page // 16) * self.tile_bytes, fill, np.uint8)

    def _tile(self, slot, h):
        page, place = divmod(int(slot), self.page)
        at = ((page * self.h_kv + h) * (self.page // 16) + place // 16) * self.tile_bytes
        return self.bytes[at:at + self.tile_bytes], place % 16

    def write(self, x, slots, which):
        """x [n][h_kv][d]; which: 0 keys, 1 values."""
        codes, s, m = quantise(x)
        d, groups = self.d, self.d // 32
        for i, slot in enumerate(slots):
            if slot < 0 or slot >= self.n_pages * self.page:
                continue
            for h in range(self.h_kv):
                tile, t = self._tile(slot, h)
                for g in range(groups):
                    c = codes[i, h, 32 * g:32 * g + 32]
                    at = which * 8 * d + (g * 16 + t) * 16
                    tile[at:at + 16] = c[0::2] | (c[1::2] << 4)
                    sb, mb = (np.array([v], np.float16).view(np.uint8) for v in (s[i, h, g], m[i, h, g]))
                    if which == 0:
                        at = 16 * d + (t * groups + g) * 4
                        tile[at:at + 2], tile[at + 2:at + 4] = sb, mb
                    else:
                        at = 18 * d + ((t // 2) * groups + g) * 8 + 2 * (t % 2)
                        tile[at:at + 2], tile[at + 4:at + 6] = sb, mb

    def read(self, slots, which):
        """fp64 values [n][h_kv][d]; zeros where the slot is outside the pool."""
        d, groups = self.d, self.d // 32
        out = np.zeros((len(slots), self.h_kv, d))
        for i, slot in enumerate(slots):
            if slot < 0 or slot >= self.n_pages * self.page:
                continue
            for h in range(self.h_kv):
                tile, t = self._tile(slot, h)
                for g in range(groups):
                    at = which * 8 * d + (g * 16 + t) * 16
                    b = tile[at:at + 16]
                    c = np.stack([b & 15, b >> 4], -1).reshape(32).astype(np.float64)
                    if which == 0:
                        at = 16 * d + (t * groups + g) * 4
                        s, m = tile[at:at + 4].copy().view(np.float16).astype(np.float64)
                    else:
                        at = 18 * d + ((t // 2) * groups + g) * 8
                        z = tile[at:at + 8].copy().view(np.float16).astype(np.float64)
                        s, m = z[t % 2], z[2 + t % 2]
                    out[i, h, 32 * g:32 * g + 32] = m + s * c
        return out


def sees(p, j, window, sinks):
    return j <= p and (window == 0 or j > p - window or j < sinks)


def attend(q, k, v, length, window, sinks, scale, hidden=()):
    """One sequence: q [n][h_q][d], k, v [length][h_kv][d] fp64.  Tokens in
    `hidden` are not seen.  Returns out [n][h_q][d], the same sums over |v|
    (what roundings of the weights and values scale with) and the largest
    scale * sum |q||k| of a row's visible tokens (what roundings of the logits
    scale with) [n][h_q]."""
    n, h_q, d = q.shape
    out, mag, lmag = np.zeros((n, h_q, d)), np.zeros((n, h_q, d)), np.zeros((n, h_q))
    group = h_q // k.shape[1]
    for i in range(n):
        p = length - n + i
        js = np.array([j for j in range(length) if sees(p, j, window, sinks) and j not in hidden], int)
        if len(js) == 0:
            continue
        for h in range(h_q):
            kk, vv = k[js, h // group], v[js, h // group]
            x = scale * (kk @ q[i, h])
            w = np.exp(x - x.max())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
            lmag[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, mag, lmag
