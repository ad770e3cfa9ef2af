"""Device functions of the paged cache's attention, each run by a small kernel of
its own (tests/native/kvp_checks.cu)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from bit_decode_selective_b200 import build

pytestmark = pytest.mark.gpu

SOURCE = os.path.join(build.ROOT, "tests", "native", "kvp_checks.cu")
LIB = os.path.join(build.ROOT, "_build", "kvp_checks.so")


@pytest.fixture(scope="module")
def checks():
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    subprocess.run([build.NVCC, *build.NVCC_FLAGS, "-shared", SOURCE, "-o", LIB], check=True)
    return ctypes.CDLL(LIB)


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("mode,waits,drains,gave_up,seconds", [
    (0, 0, 0, 0, (0, 0)),   # what it waits for has happened
    (1, 0, 2, 0, (0, 1)),   # the drain runs out: once for each of the two warps
    (2, 64, 0, 1, (1, 0)),  # the wait runs out: at most once a thread, at least once
    (3, 0, 2, 1, (0, 1)),   # after a wait has given up the next one returns at once, the drain still waits
])
def test_waits_that_run_out_are_counted(checks, mode, waits, drains, gave_up, seconds):
    counts, flag = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ns = torch.zeros(2, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    assert checks.kvp_check_wait(mode, ptr(counts), ptr(flag), ptr(ns)) == 0
    got = counts.tolist()
    assert (1 <= got[0] <= waits) if waits else got[0] == 0
    assert got[1] == drains and flag.item() == gave_up
    for t, s in zip(ns.tolist(), seconds):
        assert s * 10 ** 9 <= t <= s * 10 ** 9 + 5 * 10 ** 8


# ---------------------------------------------------------------------------
# the cut of the work

ROWS, STEP, EXTRA = {True: 8, False: 256}, {True: 2, False: 8}, {True: 8, False: 4}


def items(few, counts, lens, group, window, sinks):
    """(sequence, row tile, steps) of every row tile in the order of the line."""
    for b, (n, length) in enumerate(zip(counts, lens)):
        rows = n * group
        if rows == 0 or (rows <= 64) != few:
            continue
        for rt in range(-(-rows // ROWS[few])):
            p0 = length - n + rt * ROWS[few] // group
            p1 = length - n + (min((rt + 1) * ROWS[few], rows) - 1) // group
            lo = max(0, p0 - window + 1) if window else 0
            first = lo // 16
            sink = min(-(-min(sinks, lo) // 16), first)
            tiles = 0 if p1 < 0 else sink + p1 // 16 + 1 - first
            yield b, rt, max(1, -(-tiles // STEP[few]))


MIXED = [int(x) for x in np.random.default_rng(0).integers(0, 5000, 300)]
NEAR = 2 ** 26 - 8  # steps of an item that takes 2^26 with its fixed cost


@pytest.mark.parametrize("few,counts,lens,h_kv,group,window,sinks", [
    (True, [1], [8192], 8, 4, 0, 0),
    (True, [1] * 64, MIXED[:64], 8, 4, 0, 0),            # the last batch that every warp searches by itself
    (True, [1] * 65, MIXED[:65], 8, 4, 100, 4),          # a sequence per thread
    (True, [1] * 128, MIXED[:128], 2, 8, 0, 0),
    (True, [1] * 129, MIXED[:129], 2, 8, 0, 0),          # several sequences per thread
    (True, [i % 4 for i in range(300)], MIXED, 5, 3, 0, 0),
    (True, [9, 70, 1, 0, 64] * 60, MIXED, 1, 1, 300, 20),  # several row tiles, others' sequences between
    (False, [9, 70, 1, 0, 64] * 60, MIXED, 1, 1, 300, 20),
    (False, [3000, 1, 700], [3000, 90, 100000], 8, 4, 0, 0),
    (False, [10 ** 6, 0, 300], [10 ** 6, 7, 2 ** 30], 2, 1, 4096, 64),
    # lines of about 2^32 steps and more, which are cut in larger units, and KV
    # heads whose place on the line passes 2^32
    (True, [1] * 64, [32 * NEAR] * 63 + [32 * NEAR - 32], 1, 1, 0, 0),   # 2^32 - 1
    (True, [1] * 64, [32 * NEAR] * 63 + [32 * NEAR - 96], 1, 1, 0, 0),   # 2^32 - 3
    (True, [1] * 64, [32 * NEAR] * 64, 1, 1, 0, 0),                      # 2^32
    (True, [1], [2 ** 31 - 1024], 65, 1, 0, 0),
    (True, [1] * 200, [2 ** 31 - 1024] * 200, 65, 1, 0, 0),
    (True, [1] * 2, [2 ** 31 - 1024, 10], 65535, 1, 0, 0),
    (False, [10 ** 6], [2 ** 31 - 1024], 8, 1, 0, 0),
    (False, [300, 200], [2 ** 31 - 1024] * 2, 65535, 2, 0, 0),
])
@pytest.mark.parametrize("ctas,min_steps", [(444, 4), (148, 1)])
def test_cut_of_the_work(checks, few, counts, lens, h_kv, group, window, sinks, ctas, min_steps):
    """The ranges follow each other over the whole line, differ by a unit at most,
    and every CTA finds the item that its range starts in."""
    cu = np.concatenate([[0], np.cumsum(counts)])
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    out, cu_d, lens_d = torch.zeros(ctas, 12, dtype=torch.int64, device="cuda"), dev(cu), dev(lens)
    torch.cuda.synchronize()
    assert checks.kvp_check_range(int(few), ctas, len(counts), h_kv, group, int(cu[-1]), ptr(cu_d), ptr(lens_d),
                                  (2 ** 31 - 1) // 16, 4, window, sinks, min_steps, ptr(out)) == 0
    got = out.tolist()
    line, at = [], 0
    for b, rt, steps in items(few, counts, lens, group, window, sinks):
        line.append((at, b, rt, steps))
        at += (steps + EXTRA[few]) * h_kv
    total = at
    used = [r for r in got if r[0] < r[1]]
    assert got[:len(used)] == used and used[0][0] == 0 and used[-1][1] == total
    assert all(a[1] == b[0] for a, b in zip(used, used[1:]))
    unit = 1
    while total // unit >= 2 ** 31:
        unit *= 2
    units = -(-total // unit)
    assert len(used) == min(ctas, -(-units // min_steps))
    sizes = [u1 - u0 for u0, u1, *_ in used]
    assert max(sizes) - min(sizes[:-1] or sizes) <= unit
    starts = [s for s, *_ in line]
    for cta, (u0, u1, at, b, rt, g, steps, q0, n, length, first, last) in enumerate(used):
        s, wb, wrt, wsteps = line[int(np.searchsorted(starts, u0, "right")) - 1]
        each = wsteps + EXTRA[few]
        assert (b, rt, steps, g, at) == (wb, wrt, wsteps, (u0 - s) // each, s + (u0 - s) // each * each)
        assert (q0, n, length) == (cu[b], counts[b], lens[b])
        assert first == last == cta
