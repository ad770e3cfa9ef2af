"""Device functions of the paged cache's attention, each run by a small kernel of
its own (tests/native/kvp_checks.cu)."""
import ctypes
import os
import subprocess

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
