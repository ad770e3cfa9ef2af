"""Calls of the paged cache at the far ends of what include/sf.h allows: batches
of hundreds, contexts of 131,072 tokens, windows and page tables next to 2^31."""
import numpy as np
import pytest
import torch

from test_gpu_paged import Case, check, i32, queries

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
