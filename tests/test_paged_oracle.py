"""Pins of the paged-cache oracle, and the argument checks of the paged-cache
entry points (all on the host: nothing is launched)."""
import ctypes

import numpy as np
import pytest

from bit_decode_selective_b200 import abi
from oracle import paged

P16 = ctypes.c_void_p(16)


@pytest.fixture(scope="module")
def L():
    from bit_decode_selective_b200.build import build_library

    build_library()
    return abi.lib()


def test_quantiser_by_hand():
    # 0, 1, .., 15 twice: step 1, offset 0, every value on the grid
    x = np.arange(32.0) % 16
    q, s, m = paged.quantise(x)
    assert s[0] == 1 and m[0] == 0 and np.array_equal(q, x)
    # halves round up, the ends clamp to the grid
    x = np.array([0.0, 15.0] + [0.5, 1.5, 14.5, 14.49] + [3.0] * 26)
    q, _, _ = paged.quantise(x)
    assert list(q[:6]) == [0, 15, 1, 2, 15, 14]
    # constant groups: step 0, code 0, the value itself
    q, s, m = paged.quantise(np.full(32, -3.0))
    assert s[0] == 0 and not q.any() and np.array_equal(paged.values(q, s, m), np.full(32, -3.0))
    # NaN counts as 0, infinities as the limit; all stored values are finite in fp16
    x = np.zeros(32)
    x[:3] = [np.nan, np.inf, -np.inf]
    v = paged.stored(x)
    assert np.isfinite(v.astype(np.float16)).all() and v[1] > 65000 and v[2] < -65000
    # the stored value is within half a step, plus the roundings of s (15 half
    # steps of fp16 at most) and m
    rng = np.random.default_rng(0)
    x = rng.normal(size=(50, 128))
    q, s, m = paged.quantise(x)
    err = np.abs(paged.values(q, s, m) - x).reshape(50, 4, 32).max(-1)
    assert (err <= s.astype(float) * (0.5 + 15 * 2.0 ** -11) + np.abs(m.astype(float)) * 2.0 ** -11).all()


def test_pool_bytes_by_hand():
    pool = paged.Pool(2, 16, 2, 64)
    x = np.zeros((1, 2, 64))
    x[0, 1, :32] = np.arange(32) % 16           # group 0 of head 1: s = 1, m = 0
    x[0, 1, 32:] = 2 * (np.arange(32) % 16) - 4  # group 1: s = 2, m = -4
    slot = 16 + 5                                # page 1, token 5
    pool.write(x, [slot], 0)
    pool.write(x, [slot], 1)
    tile = pool.bytes.reshape(2, 2, 1, 1280)[1, 1, 0]
    nib = np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2, np.uint8)
    want = np.zeros(1280, np.uint8)
    for base in (0, 512):
        for g in (0, 1):
            want[base + (g * 16 + 5) * 16:][:16] = nib
    f16 = lambda *v: np.array(v, np.float16).view(np.uint8)
    want[1024 + (5 * 2) * 4:][:8] = f16(1, 0, 2, -4)
    want[1152 + (2 * 2) * 8:][:16] = f16(0, 1, 0, 0, 0, 2, 0, -4)  # pair 2: (s4, s5, m4, m5) per group
    assert np.array_equal(tile, want)
    assert np.array_equal(pool.read([slot], 0)[0, 1], x[0, 1])
    assert np.array_equal(pool.read([slot], 1)[0, 1], x[0, 1])
    assert not pool.read([-1, 32], 0).any()


def test_pool_round_trip():
    rng = np.random.default_rng(1)
    pool = paged.Pool(3, 32, 2, 128, fill=255)
    slots = rng.permutation(96)[:40]
    x = rng.normal(size=(40, 2, 128))
    pool.write(x, slots, 0)
    pool.write(2 * x, slots, 1)
    assert np.array_equal(pool.read(slots, 0), paged.stored(x))
    assert np.array_equal(pool.read(slots, 1), paged.stored(2 * x))


def test_attend_against_closed_forms():
    rng = np.random.default_rng(2)
    k, v, q = rng.normal(size=(40, 2, 64)), rng.normal(size=(40, 2, 64)), rng.normal(size=(3, 4, 64))
    full, _, _ = paged.attend(q, k, v, 40, 0, 0, 0.125)
    # a window of everything is no window; the last query sees all tokens
    same, _, _ = paged.attend(q, k, v, 40, 40, 0, 0.125)
    assert np.array_equal(full, same)
    x = 0.125 * k[:, 1] @ q[2, 3]
    assert np.allclose(full[2, 3], np.exp(x) @ v[:, 1] / np.exp(x).sum(), rtol=1e-12)
    # window 1 without sinks: the query's own token
    own, _, _ = paged.attend(q, k, v, 40, 1, 0, 0.125)
    assert np.allclose(own[1, 0], v[38, 0])
    # window 1, one sink: two tokens
    two, _, _ = paged.attend(q, k, v, 40, 1, 1, 0.0)
    assert np.allclose(two[0, 2], (v[0, 1] + v[37, 1]) / 2)
    # a query before the first token sees nothing
    none, _, _ = paged.attend(q, k[:2], v[:2], 2, 0, 0, 1.0)
    assert not none[0].any() and none[1].any()


# ---------------------------------------------------------------------------
# refusals


def kvp(n_pages=4, page=16, h_kv=2, d=128, pool=16):
    return abi.sf_kvp(n_pages, page, h_kv, d, pool)


def test_bytes(L):
    n = ctypes.c_size_t()
    assert abi.sf_kvp_bytes(10, 64, 8, 128, ctypes.byref(n)) == 0 and n.value == 10 * 64 * 8 * 160
    assert abi.sf_kvp_bytes(10, 16, 1, 64, ctypes.byref(n)) == 0 and n.value == 10 * 16 * 80
    assert abi.sf_kvp_bytes(10, 64, 8, 128, None) == abi.SF_ERR_INVALID_ARG


@pytest.mark.parametrize("bad,status", [
    (dict(d=96), abi.SF_ERR_UNSUPPORTED), (dict(page=8), abi.SF_ERR_UNSUPPORTED), (dict(page=48), abi.SF_ERR_UNSUPPORTED),
    (dict(page=2048), abi.SF_ERR_UNSUPPORTED), (dict(n_pages=0), abi.SF_ERR_INVALID_ARG),
    (dict(h_kv=0), abi.SF_ERR_INVALID_ARG), (dict(n_pages=1 << 27), abi.SF_ERR_UNSUPPORTED),
    (dict(pool=None), abi.SF_ERR_INVALID_ARG), (dict(pool=24), abi.SF_ERR_INVALID_ARG)])
def test_descriptor_refusals(L, bad, status):
    kv = ctypes.byref(kvp(**bad))
    assert abi.sf_kvp_write(kv, P16, 256, 128, P16, 256, 128, 0, 1, P16, None, None) == status
    assert abi.sf_kvp_read(kv, P16, 1, P16, P16, 0, None, None) == status
    assert abi.sf_kvp_attend(kv, P16, 512, 128, 0, 1, None, P16, 1, P16, 1, 4, 1.0, 0, 0, P16, None, P16, 1 << 30,
                             None) == status
    assert abi.sf_last_error()


def test_write_and_read_refusals(L):
    kv = ctypes.byref(kvp())
    bad = abi.SF_ERR_INVALID_ARG
    w = lambda k=P16, kr=256, kh=128, v=P16, vr=256, vh=128, t=0, n=1, s=P16, e=None: abi.sf_kvp_write(
        kv, k, kr, kh, v, vr, vh, t, n, s, e, None)
    assert w(t=3) == bad and w(t=-1) == bad and w(n=-1) == bad and w(s=None) == bad
    assert w(s=ctypes.c_void_p(18)) == bad and w(e=ctypes.c_void_p(18)) == bad
    assert w(k=ctypes.c_void_p(24)) == bad and w(v=ctypes.c_void_p(24)) == bad
    assert w(kr=257) == bad and w(vh=4) == bad and w(kh=-128) == bad
    assert w(n=0) == 0 and w(k=None, v=None) == 0  # nothing to do
    r = lambda s=P16, n=1, k=P16, v=P16, t=0, e=None: abi.sf_kvp_read(kv, s, n, k, v, t, e, None)
    assert r(t=3) == bad and r(n=-1) == bad and r(s=None) == bad and r(k=ctypes.c_void_p(24)) == bad
    assert r(n=0) == 0 and r(k=None, v=None) == 0
    # fp32 rows: a stride of 4 elements is 16 bytes
    assert w(t=2, n=0, kr=260, kh=132) == 0


def test_attend_refusals(L):
    d = kvp()
    kv = ctypes.byref(d)
    bad, uns = abi.SF_ERR_INVALID_ARG, abi.SF_ERR_UNSUPPORTED

    def at(q=P16, row=512, head=128, t=0, n=2, cu=None, pages=P16, mp=2, lens=P16, batch=2, hq=4, scale=0.1, window=0,
           sinks=0, out=P16, e=None, ws=P16, nb=1 << 40):
        return abi.sf_kvp_attend(kv, q, row, head, t, n, cu, pages, mp, lens, batch, hq, scale, window, sinks, out, e,
                                 ws, nb, None)

    assert at(t=2) == uns and at(t=5) == bad
    assert at(batch=0) == bad and at(n=-1) == bad and at(hq=3) == bad and at(hq=0) == bad
    assert at(n=3) == bad  # no cu_q and not a multiple of batch
    assert at(scale=float("nan")) == bad and at(scale=float("inf")) == bad
    assert at(window=-1) == bad and at(sinks=-1) == bad
    assert at(mp=0) == bad and at(mp=1 << 28) == uns
    assert at(pages=None) == bad and at(lens=None) == bad and at(cu=ctypes.c_void_p(18)) == bad
    assert at(pages=ctypes.c_void_p(18)) == bad and at(e=ctypes.c_void_p(18)) == bad
    assert at(q=None) == bad and at(out=None) == bad and at(q=ctypes.c_void_p(24)) == bad
    assert at(row=516) == bad and at(head=4) == bad and at(row=-512) == bad
    assert at(batch=70000, n=70000) == uns and at(n=1 << 30, batch=1) == uns
    assert at(n=0) == 0  # no queries: nothing to do
    need = abi.sf_kvp_attend_workspace_bytes(kv, 2, 2, 4)
    if need:
        assert at(nb=need - 1) == abi.SF_ERR_WORKSPACE and at(ws=None) == abi.SF_ERR_WORKSPACE
        assert at(ws=ctypes.c_void_p(24)) == bad
    assert abi.sf_kvp_attend_workspace_bytes(kv, 2, 0, 4) == 0
    assert abi.sf_kvp_attend_workspace_bytes(None, 2, 2, 4) == 0
