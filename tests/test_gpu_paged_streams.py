"""Calls of the paged cache on several streams at once, with nothing between them
but what their arguments need."""
import numpy as np
import pytest
import torch

from test_gpu_paged import Case, check, i32, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq", [1, 40])
def test_overlapping_calls(nq):
    """Calls in turn on the current stream and on another one, whose default
    workspaces and outputs are of one size.  The second stream's inputs are ready
    long before, so nothing else orders the two."""
    d, h_kv = 128, 2
    case = Case(41, [3000, 2500], h_kv, d, 64)
    q, cu = queries(case, [nq, nq], 8, "fp16")
    args = (i32(case.pages), i32(case.lens))
    slots = i32(case.pages[0, np.arange(2000) // 64] * 64 + np.arange(2000) % 64)
    want = case.cache.attend(q, *args)
    want_kv = case.cache.read(slots)
    if nq == 1:
        check(case, want, q, cu, "fp16", 0, 0, d ** -0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        outs, kvs = [], []
        for i in range(20):
            stream = side if i % 2 else None
            outs.append(case.cache.attend(q, *args, stream=stream))
            kvs.append(case.cache.read(slots, stream=stream))
            torch.full_like(want, 3.0)  # memory that changes hands on the current stream
        torch.cuda.synchronize()
        for out, (k, v) in zip(outs, kvs):
            assert torch.equal(out, want) and torch.equal(k, want_kv[0]) and torch.equal(v, want_kv[1])


def test_memory_given_back_on_the_current_stream_is_not_taken():
    """A block that the current stream has just freed does not become the memory of a call on another one."""
    case = Case(43, [100], 2, 64, 16)
    q, _ = queries(case, [1], 8, "fp16")
    args = (i32(case.pages), i32(case.lens))
    slots = i32(case.pages[0, np.arange(100) // 16] * 16 + np.arange(100) % 16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda: [case.cache.attend(q, *args, stream=side)], lambda: case.cache.read(slots, stream=side)):
        held = call()  # of the sizes that the call allocates
        free = [torch.empty_like(t) for t in held for _ in range(4)]
        given_back = {t.data_ptr() for t in free}
        del free
        assert not given_back & {t.data_ptr() for t in call()}
        del held
    torch.cuda.synchronize()


@pytest.mark.parametrize("nq", [1, 40])
def test_arguments_may_be_dropped(nq):
    """Temporaries given to a call on another stream are not overwritten before it has read them."""
    case = Case(45, [3000, 2500], 2, 128, 64)
    q, _ = queries(case, [nq, nq], 8, "fp16")
    pages, lens = i32(case.pages), i32(case.lens)
    want = case.cache.attend(q, pages, lens)
    side = torch.cuda.Stream()
    for _ in range(5):
        outs = []
        for _ in range(10):
            temp, p, n = q.clone(), pages.clone(), lens.clone()
            side.wait_stream(torch.cuda.current_stream())
            outs.append(case.cache.attend(temp, p, n, stream=side))
            del temp, p, n
            for like in (q, pages, lens):
                torch.full_like(like, 7)  # takes what was given back
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in outs)


def test_side_stream_inside_a_capture():
    """A call on a stream that a capture has forked to, its memory from the capture's own."""
    case = Case(47, [300], 2, 64, 16)
    q, _ = queries(case, [1], 8, "bf16")
    args = (i32(case.pages), i32(case.lens))
    want = case.cache.attend(q, *args)
    side = torch.cuda.Stream()
    qq, out = torch.zeros_like(q), torch.empty_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        a = case.cache.attend(qq + 0, *args, stream=side)
        b = case.cache.attend(qq, *args)
        torch.cuda.current_stream().wait_stream(side)
        out.copy_(a)
    for x in (q, -q, q):
        qq.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, case.cache.attend(x, *args)) and torch.equal(b, out)
    assert torch.equal(out, want)
