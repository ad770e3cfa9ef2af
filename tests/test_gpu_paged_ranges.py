"""Calls of the paged cache at the far ends of what include/sf.h allows: batches
of hundreds, contexts of 131,072 tokens, windows and page tables next to 2^31."""
import numpy as np
import pytest
import torch

from test_gpu_paged import Case, check, i32, queries, spot_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,n", [(32, 10), (200, 50)])
@pytest.mark.parametrize("sinks", [0, 40])
def test_huge_window_with_queries_before_the_sequence(nq, n, sinks):
    """More queries than tokens, so that the first stand before the sequence, and a
    window of nearly 2^31 tokens: position minus window passes -2^31 for rows that
    share a tile with rows that see something, and the window hides nothing."""
    page, d = 16, 64
    case = Case(51, [n], 1, d, page)
    q, cu = queries(case, [nq], 1, "fp16")
    table = torch.full((1, (2 ** 31 - 1) // page), -1, dtype=torch.int32, device="cuda")
    table[0, :case.pages.shape[1]] = i32(case.pages[0])
    window = table.shape[1] * page - 1
    assert n - nq - window + 1 < -2 ** 31
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = case.cache.attend(q, table, i32([n]), window=window, sinks=sinks, bad=bad)
    check(case, out, q, cu, "fp16", 0, 0, d ** -0.5)
    assert torch.equal(out, case.cache.attend(q, i32(case.pages), i32([n]))) and bad.item() == 0


@pytest.mark.parametrize("batch,window", [(129, 0), (300, 50), (1000, 0)])
def test_batches_of_hundreds(batch, window):
    """Single tokens, drafts and idle sequences; several sequences per thread of the place search."""
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 400, batch)]
    case = Case(batch, lens, 2, 64, 16)
    q, cu = queries(case, [1] * batch, 8, "fp16")
    out = case.cache.attend(q, i32(case.pages), i32(lens), window=window, sinks=2)
    assert torch.equal(out, case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu), window=window, sinks=2))
    rows = [(int(b), 0) for b in rng.integers(0, batch, 40)] + [(batch - 1, 0), (128, 0)]
    spot_check(case, out, q, cu, "fp16", window, 2, rows)
    counts = rng.integers(0, 4, batch)
    counts[batch // 2] = 90  # a chunk among them
    q, cu = queries(case, counts, 8, "fp16")
    out = case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu), window=window, sinks=2)
    rows = [(int(b), int(counts[b]) - 1) for b in rng.integers(0, batch, 40) if counts[b]] + [(batch // 2, 0), (batch // 2, 89)]
    spot_check(case, out, q, cu, "fp16", window, 2, rows)


@pytest.mark.parametrize("counts", [[1, 1], [7, 2], [100, 1], [2048, 300]])
def test_contexts_of_131072_tokens(counts):
    """Lengths at which the cases are measured, odd ones, both kernels."""
    lens = [131073, 70001]
    case = Case(53, lens, 1, 128, 64)
    q, cu = queries(case, counts, 4, "fp16", 2.0)
    out = case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu))
    spot_check(case, out, q, cu, "fp16", 0, 0, [(b, r) for b, n in enumerate(counts) for r in {0, n // 2, n - 1}])
    out = case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu), window=33000, sinks=5)
    spot_check(case, out, q, cu, "fp16", 33000, 5, [(b, r) for b, n in enumerate(counts) for r in {0, n - 1}])
