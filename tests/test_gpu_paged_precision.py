"""The few-row attention of the paged cache held to the bound that its exact products
allow (paged_bounds.py), also beside sequences of the many-row kernel."""
import numpy as np
import pytest
import torch

from bit_decode_selective_b200.ops import PagedKVCache
from oracle import paged
from paged_bounds import few_row_bound, tied_by_offsets
from test_gpu_paged import f64, i32, rounded, tokens

pytestmark = pytest.mark.gpu


class Sequences:
    """Tokens given as k, v [length][h_kv][d] per sequence, in shuffled pages."""

    def __init__(self, rng, k, v, page):
        h_kv, d = k[0].shape[1:]
        self.lens = [len(x) for x in k]
        counts = [-(-n // page) for n in self.lens]
        order = rng.permutation(sum(counts) + 1)
        self.pages = np.zeros((len(k), max(counts)), np.int64)
        self.cache = PagedKVCache(len(order), page, h_kv, d)
        self.k_raw, self.k, self.v = [], [], []
        for b, (kb, vb) in enumerate(zip(k, v)):
            mine, order = order[:counts[b]], order[counts[b]:]
            self.pages[b, :counts[b]] = mine
            j = np.arange(len(kb))
            kd, vd = rounded(kb, "fp16"), rounded(vb, "fp16")
            self.cache.write(kd, vd, i32(mine[j // page] * page + j % page))
            self.k_raw.append(f64(kd)), self.k.append(paged.stored(f64(kd))), self.v.append(paged.stored(f64(vd)))

    def check(self, out, q, cu, dtype, window, sinks, scale, most=10 ** 9):
        """Every sequence of at most `most` queries."""
        got, qh = f64(out), f64(q)
        for b, n in enumerate(self.lens):
            rows = slice(cu[b], cu[b + 1])
            if not 0 < cu[b + 1] - cu[b] <= most:
                continue
            ref, tol = few_row_bound(dtype, qh[rows], self.k_raw[b], self.k[b], self.v[b], n, window, sinks, scale)
            err = np.abs(got[rows] - ref)
            assert (err <= tol).all(), (b, float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:5])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("group", [1, 8, 13, 20, 32])  # up to four columns of eight rows
@pytest.mark.parametrize("d", [64, 128])
def test_logits_that_offsets_decide(dtype, group, d):
    rng = np.random.default_rng(group)
    h_kv, lens = 2, [300, 17, 1000]
    q = rng.uniform(0.5, 1.5, (len(lens), h_kv, 1, d))
    q = rounded(np.broadcast_to(q, (len(lens), h_kv, group, d)).reshape(len(lens), h_kv * group, d), dtype)
    first = f64(q).reshape(len(lens), h_kv, group, d)[:, :, 0]
    seqs = Sequences(rng, [tied_by_offsets(rng, n, h_kv, d, first[b]) for b, n in enumerate(lens)],
                     [rng.normal(size=(n, h_kv, d)) for n in lens], 16)
    out = seqs.cache.attend(q, i32(seqs.pages), i32(lens))
    # the heads of a KV head have one query: one of them is enough for the oracle
    for h in (0, group - 1):
        pick = [h, group + h]
        seqs.check(out[:, pick], q[:, pick], range(len(lens) + 1), dtype, 0, 0, d ** -0.5)


@pytest.mark.parametrize("gain", [1.0, 20.0])
@pytest.mark.parametrize("counts,h_kv,group,d,window,sinks", [
    ([1, 1, 1], 2, 4, 128, 0, 0),
    ([1, 1, 1], 1, 8, 64, 100, 4),
    ([5, 1, 3], 2, 4, 64, 0, 0),
    ([5, 5, 5], 1, 12, 128, 33, 3),      # 60 rows
    ([1, 100, 2], 2, 4, 128, 0, 0),      # beside a sequence of the many-row kernel
    ([16, 17, 1], 1, 4, 64, 50, 0),      # 64 rows and 68
])
def test_few_rows(gain, counts, h_kv, group, d, window, sinks):
    rng = np.random.default_rng(sum(counts))
    lens = [777, 130, 64]
    seqs = Sequences(rng, [tokens(rng, n, h_kv, d) for n in lens], [rng.normal(size=(n, h_kv, d)) for n in lens], 32)
    cu = np.concatenate([[0], np.cumsum(counts)])
    q = rounded(rng.normal(size=(cu[-1], h_kv * group, d)) * gain, "fp16")
    out = seqs.cache.attend(q, i32(seqs.pages), i32(lens), cu_q=i32(cu), window=window, sinks=sinks)
    seqs.check(out, q, cu, "fp16", window, sinks, d ** -0.5, most=64 // group)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nq", [1, 80])
def test_values_at_the_limit(dtype, nq):
    """Values and keys beyond the largest that is stored: fp16 outputs stay finite, as
    weights rounded up make 65,472 (1 + 2^-11) at most."""
    rng = np.random.default_rng(nq)
    n, d = 200, 128
    k = rng.choice([-1.0, 1.0], (n, 1, d)) * 7e4
    v = np.full((n, 1, d), 7e4)
    v[:, :, 1::2] *= -1
    v[:, :, 64:] = 65408 - rng.integers(0, 2, (n, 1, 64)) * 1000.0
    cache = PagedKVCache(13, 16, 1, d)
    cache.write(rounded(k, "fp32"), rounded(v, "fp32"), i32(np.arange(n)))
    ks, vs = paged.stored(k.astype(np.float32).astype(float)), paged.stored(v.astype(np.float32).astype(float))
    q = rounded(rng.normal(size=(nq, 4, d)) * 1e-4, dtype)
    out = cache.attend(q, i32(np.arange(13)[None]), i32([n]))
    ref, mag, lmag = paged.attend(f64(q), ks, vs, n, 0, 0, d ** -0.5)
    # keys rounded to fp16 too, as the many-row kernel does
    delta = lmag * (2.0 ** -11 + 2.0 ** -16) + (lmag + 2) * 2.0 ** -19
    half = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8
    tol = (np.abs(ref) * half + mag * (2.0 ** -10 + np.expm1(2 * delta)[..., None] + (n / 16 + 8) * 17 * 2.0 ** -23)) * (1 + 2.0 ** -6)
    got = f64(out)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()
