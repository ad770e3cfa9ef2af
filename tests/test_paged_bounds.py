"""The bound of the few-row attention tells right from wrong: mistakes planted in
the oracle's logits pass it, the oracle in fp32 stays far within."""
import numpy as np
import pytest

from oracle import paged
from paged_bounds import few_row_bound, tied_by_offsets


def attend(q, logits, v):
    w = np.exp(logits - logits.max())
    return (w / w.sum()) @ v


@pytest.mark.parametrize("d", [64, 128])
def test_mistakes_in_the_group_sums_show(d):
    rng = np.random.default_rng(d)
    n, scale = 300, d ** -0.5
    q = rng.uniform(0.5, 1.5, (1, 1, d)).astype(np.float16).astype(float)
    k_raw = tied_by_offsets(rng, n, 1, d, q[0]).astype(np.float16).astype(float)
    k, v = paged.stored(k_raw), paged.stored(rng.normal(size=(n, 1, d)))
    ref, tol = few_row_bound("fp16", q, k_raw, k, v, n, 0, 0, scale)
    worst = lambda logits: (np.abs(attend(q, logits, v[:, 0]) - ref[0, 0]) / tol[0, 0]).max()
    x = scale * k[:, 0] @ q[0, 0]
    assert worst(x) < 1e-6 and worst(x.astype(np.float32).astype(float)) < 0.1
    _, _, m = paged.quantise(k_raw)
    sums = q[0, 0].reshape(-1, 32).sum(-1)
    m = m[:, 0].astype(float)
    high = sums.astype(np.float16).astype(float)         # the low half of the split left out
    coarse = np.round(sums * 4) / 4                      # 8 bits
    assert worst(x + scale * m @ (high - sums)) > 2
    assert worst(x + scale * m @ (coarse - sums)) > 10
    assert worst(x + scale * m @ np.eye(len(sums))[0] * 2.0 ** -6) > 2  # one group's sum off by 2^-11 of itself
