"""How far the few-row attention of the paged cache (at most 64 rows, queries x
query heads per KV head) may be from the fp64 oracle, and inputs whose answer
hangs on its logits.

A key is m + s c, and the kernel sums s c and m apart, so with
  M = scale * sum |q| (|m| + s c)      X = the largest |logit|
a logit is off by at most
  - products and fp32 sums: 126 roundings of 2^-24 of M: the codes' products 68 (two
    steps of 16 products, 17 roundings of 2^-23 each), the offsets' 34, the sums of
    q over a group 10 and their split in two fp16 4, the factors 10: 2^-17 M;
  - q as fp16 scaled to a largest element of 2^10 or more: exact but for
    elements that become subnormal, 2^-31 of the largest each;
  - the exponent, its reference and ten moves of the reference: 2^-19 (X + 2).
Call that delta: weights and their sum each change by at most exp(delta) - 1.
Then, relative to sum p |v|:
  - weights and values as fp16: 2^-11 each (subnormal: 2^-34 of the largest
    weight, 2^-25 of a value);
  - fp32 sums over tiles of 16 tokens: 17 roundings of 2^-23 each;
and the output's own half step."""
import numpy as np

from oracle import paged

HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp16": 2.0 ** -24, "bf16": 2.0 ** -133}


def few_row_bound(dtype, q, k_raw, k, v, length, window, sinks, scale):
    """q [n][h_q][d], k_raw as written and k, v as stored [length][h_kv][d], all fp64:
    (oracle's output, how far from it the kernel may be), [n][h_q][d]."""
    n, h_q, d = q.shape
    codes, s, m = paged.quantise(k_raw)
    wide = np.abs(m.astype(float))[..., None] + s.astype(float)[..., None] * codes.reshape(*s.shape, 32)
    wide = wide.reshape(k.shape)
    group = h_q // k.shape[1]
    ref, mag, _ = paged.attend(q, k, v, length, window, sinks, scale)
    tol = np.zeros_like(ref)
    for i in range(n):
        p = length - n + i
        js = [j for j in range(length) if paged.sees(p, j, window, sinks)]
        if not js:
            continue
        for h in range(h_q):
            g, a = h // group, np.abs(q[i, h])
            big = abs(scale) * (wide[js, g] @ a).max()
            small = abs(scale) * wide[js, g].sum(-1).max() * a.max() * 2.0 ** -31
            top = abs(scale) * np.abs(k[js, g] @ q[i, h]).max()
            delta = big * 2.0 ** -17 + small + (top + 2) * 2.0 ** -19
            tol[i, h] = (np.abs(ref[i, h]) * HALF[dtype]
                         + mag[i, h] * (2.0 ** -10 + np.expm1(2 * delta) + (len(js) / 16 + 8) * 17 * 2.0 ** -23)
                         + 2.0 ** -24 + len(js) * np.abs(v).max() * 2.0 ** -33) * (1 + 2.0 ** -6) + TINY[dtype]
    return ref, tol


def tied_by_offsets(rng, length, h_kv, d, q):
    """Keys for one query's heads (all elements of q positive, the same for the heads of a
    KV head) whose logits tie at about 280 * sqrt(d / 128): each token has a large offset in
    one of its groups, so that only the product of offsets and group sums tells
    the tokens' weights."""
    k = rng.normal(size=(length, h_kv, d))
    groups = d // 32
    sums = q.reshape(h_kv, groups, 32).sum(-1)
    for j in range(length):
        g = rng.integers(groups)
        k[j, :, 32 * g:32 * g + 32] += (100 * 32 / sums[:, g])[:, None]
    return k
