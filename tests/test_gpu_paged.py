"""The paged 4-bit KV cache on the GPU against the fp64 oracle (oracle/paged.py).

Codes and grids are bit-exact.  Values read back are m + s q rounded to fp32 and
then to the type: half a step of each.  Attention outputs are held, element by
element, to the sum of the roundings the entry point may make:
  - the output: half a step of its type;
  - keys, values and softmax weights as fp16 operands: 2^-11 each, the keys' on
    the logit (2^-11 scale sum |q||k| =: delta, so weights move by at most
    exp(2 delta) - 1), the others on sum p |v|;
  - fp16 subnormals: 2^-25 absolute on a key or value, 2^-33 of the largest
    weight on a weight;
  - fp32 sums: 2^-18 of the same magnitudes.
"""
import ctypes

import numpy as np
import pytest
import torch

from bit_decode_selective_b200 import abi
from bit_decode_selective_b200.ops import PagedKVCache
from oracle import paged

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
# smallest step of each type (subnormal spacing)
TINY = {"fp16": 2.0 ** -24, "bf16": 2.0 ** -133, "fp32": 2.0 ** -149}


def f64(t):
    return t.double().cpu().numpy()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def rounded(x, dtype):
    """x on the type's grid, as a device tensor."""
    return torch.from_numpy(x.copy()).to(DT[dtype]).cuda()


def tokens(rng, n, h, d):
    k = rng.normal(size=(n, h, d))
    k[:, :, rng.permutation(d)[:4]] *= 10
    return k


def special(rng, n, h, d):
    x = rng.normal(size=(n, h, d))
    x[0, 0, :32] = 0.25                            # constant
    if n > 1:
        x[1, 0, :32] = np.linspace(-1, 1, 32)      # borders
        x[1, 0, 32:64] = np.arange(32) / 2         # exact halves of a step
    if n > 2:
        x[2, 0, :32] = 0.0
        x[2, 0, :2] = [-0.0, 0.0]
        x[2, 0, 32:64] *= 1e-7                      # step rounds to a subnormal or to 0
    if n > 3:
        x[3, 0, :3] = [np.nan, np.inf, -np.inf]
        x[3, 0, 32:64] = np.nan
        x[3, -1, :32] *= 3e4                        # beyond the limit
    if n > 4:
        x[4, 0, :32] = rng.integers(-8, 8, 32)      # 16 levels
        x[4, 0, 32:64] = 1000 + rng.normal(size=32) * 1e-2
    return x


def grids(pool, n_pages, page, h, d):
    """(code bytes, grids as float) of pool bytes, for comparison."""
    t = np.asarray(pool).reshape(n_pages, h, page // 16, 20 * d)
    return t[..., :16 * d], t[..., 16 * d:].copy().view(np.float16).astype(np.float64)


# ---------------------------------------------------------------------------
# write and read


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,h,d,page", [(1, 8, 128, 16), (7, 1, 64, 16), (61, 5, 128, 32), (100, 2, 64, 256), (333, 3, 128, 64)])
def test_write_is_bit_exact(dtype, n, h, d, page):
    rng = np.random.default_rng(n)
    n_pages = -(-n // page) + 2
    k, v = rounded(special(rng, n, h, d), dtype), rounded(special(rng, n, h, d)[::-1], dtype)
    slots = rng.permutation(n_pages * page)[:n]
    cache = PagedKVCache(n_pages, page, h, d)
    cache.pool.fill_(0xFF)
    cache.write(k, v, i32(slots))
    want = paged.Pool(n_pages, page, h, d, fill=0xFF)
    want.write(f64(k), slots, 0)
    want.write(f64(v), slots, 1)
    got, exp = grids(cache.pool.cpu(), n_pages, page, h, d), grids(want.bytes, n_pages, page, h, d)
    assert np.array_equal(got[0], exp[0])
    assert np.array_equal(got[1], exp[1], equal_nan=True)
    for out in ("fp16", "bf16", "fp32"):
        kk, vv = cache.read(i32(slots), DT[out])
        for a, which in ((kk, 0), (vv, 1)):
            ref = want.read(slots, which)
            # one rounding to fp32, one to the type
            tol = np.abs(ref) * (HALF[out] * (1 + 2.0 ** -20) + 2.0 ** -24) + TINY[out]
            assert (np.abs(f64(a) - ref) <= tol).all()


def test_write_borders_bit_exact():
    """Many values on and next to the borders between codes."""
    rng = np.random.default_rng(5)
    n, h, d = 4096, 2, 128
    for dtype in ("fp16", "fp32"):
        s = 2.0 ** rng.integers(-6, 6, (n, h, d // 32, 1)) * (1 + rng.integers(0, 64, (n, h, d // 32, 1)) / 64)
        m = rng.normal(size=s.shape) * 3
        q = rng.integers(0, 16, (n, h, d // 32, 32)) + rng.choice([-0.5, 0.0, 0.5], (n, h, d // 32, 32))
        x = (m + s * np.clip(q, 0, 15)).reshape(n, h, d)
        x = x * (1 + rng.choice([0, 2.0 ** -22, -2.0 ** -22, 2.0 ** -12], x.shape))
        k = rounded(x, dtype)
        cache = PagedKVCache(n // 64, 64, h, d)
        cache.write(k, None, i32(np.arange(n)))
        codes, _, _ = paged.quantise(f64(k))
        t = cache.pool.cpu().numpy().reshape(n // 64, h, 4, 20 * d)[..., :8 * d].reshape(n // 64, h, 4, d // 32, 16, 16)
        t = t.transpose(0, 2, 4, 1, 3, 5).reshape(n, h, d // 2)  # token-major
        assert np.array_equal(t, codes[..., 0::2] | (codes[..., 1::2] << 4))


def test_write_padding_strides_and_bad_slots():
    rng = np.random.default_rng(6)
    n, h_q, h, d, page, n_pages = 37, 6, 3, 64, 16, 5
    qkv = rounded(rng.normal(size=(n + 2, (h_q + 2 * h) * d)), "bf16")
    rows = qkv[1:n + 1]  # views: rows and heads strided
    k = rows[:, h_q * d:(h_q + h) * d].unflatten(1, (h, d))
    v = rows[:, (h_q + h) * d:].unflatten(1, (h, d)).flip(0).contiguous().flip(0)  # another layout
    v = v if all(s >= 0 for s in v.stride()) else v.contiguous()
    slots = rng.permutation(n_pages * page)[:n].astype(np.int64)
    slots[[0, 5, 36]] = -1
    slots[7], slots[8], slots[9] = n_pages * page, -2, 2 ** 31 - 1
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = PagedKVCache(n_pages, page, h, d)
    cache.write(k, v, i32(slots), bad=bad)
    want = paged.Pool(n_pages, page, h, d)
    want.write(f64(k), slots, 0)
    want.write(f64(v), slots, 1)
    assert np.array_equal(grids(cache.pool.cpu(), n_pages, page, h, d)[0], grids(want.bytes, n_pages, page, h, d)[0])
    assert bad.item() == 3
    kk, vv = cache.read(i32(slots), torch.float32, bad=bad)
    assert bad.item() == 6
    hole = (slots < 0) | (slots >= n_pages * page)
    assert not f64(kk)[hole].any() and not f64(vv)[hole].any()
    assert np.allclose(f64(kk), want.read(slots, 0), rtol=2.0 ** -23, atol=0)
    # heads interleaved with other data: head stride larger than d
    wide = rounded(rng.normal(size=(n, h, 2 * d)), "fp16")
    cache.write(wide[:, :, d:], None, i32(np.arange(n)))
    assert np.array_equal(f64(cache.read(i32(np.arange(n)), torch.float32)[0]).astype(np.float32),
                          paged.stored(f64(wide[:, :, d:])).astype(np.float32))
    # the same slots read twice and in any order
    twice = np.concatenate([np.arange(n)[::-1], [3, 3, 3]])
    a, _ = cache.read(i32(twice))
    b, _ = cache.read(i32(np.arange(n)))
    assert torch.equal(a, b[torch.from_numpy(twice.copy()).cuda()])
    # nothing to do
    empty = torch.empty(0, h, d, dtype=torch.float16, device="cuda")
    cache.write(empty, empty, i32([]))
    assert cache.read(i32([]))[0].shape == (0, h, d)


def test_slots_that_several_tokens_name_touch_nothing_else():
    """The slot's own bytes are unspecified then; its neighbours keep theirs."""
    rng = np.random.default_rng(7)
    h, d, page = 2, 128, 16
    cache = PagedKVCache(4, page, h, d)
    x = rounded(rng.normal(size=(64, h, d)), "fp16")
    cache.write(x, x, i32(np.arange(64)))
    before = cache.read(i32(np.arange(64)))
    cache.write(x[:9], x[:9], i32([17] * 9))
    after = cache.read(i32(np.arange(64)))
    keep = [i for i in range(64) if i != 17]
    for a, b in zip(before, after):
        assert torch.equal(a[keep], b[keep])


# ---------------------------------------------------------------------------
# attention


class Case:
    """A pool with shuffled pages holding the sequences' tokens, everything else
    poisoned with NaN grids."""

    def __init__(self, seed, lens, h_kv, d, page, spread=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.h_kv, self.d, self.page = lens, h_kv, d, page
        counts = [-(-n // page) for n in lens]
        self.n_pages = sum(counts) + 2
        order = rng.permutation(self.n_pages)
        self.pages = np.full((len(lens), max(max(counts), 1) + 1), -1, np.int64)
        slots, at = [], 0
        for b, (c, n) in enumerate(zip(counts, lens)):
            self.pages[b, :c] = order[at:at + c]
            at += c
            j = np.arange(n)
            slots.append(self.pages[b, j // page] * page + j % page)
        total = sum(lens)
        k, v = tokens(rng, total, h_kv, d), rng.normal(size=(total, h_kv, d)) * spread
        self.cache = PagedKVCache(self.n_pages, page, h_kv, d)
        self.cache.pool.fill_(0xFF)
        k, v = rounded(k, "fp16"), rounded(v, "fp16")
        if total:
            self.cache.write(k, v, i32(np.concatenate(slots)))
        split = np.cumsum(lens)[:-1]
        self.k, self.v = (np.split(paged.stored(f64(x)) if total else np.zeros((0, h_kv, d)), split) for x in (k, v))
        self.rng = rng


def tolerance(dtype, ref, mag, lmag, q, scale, vmax, length):
    delta = lmag * (2.0 ** -11 + 2.0 ** -18) + abs(scale) * np.abs(q).sum(-1) * 2.0 ** -25
    weights = np.expm1(2 * delta)[..., None]
    return (np.abs(ref) * HALF[dtype] * (1 + 2.0 ** -8) + mag * (2 * 2.0 ** -11 + weights + 2.0 ** -18) * (1 + 2.0 ** -6)
            + 2.0 ** -24 + length * vmax * 2.0 ** -33 + TINY[dtype])


def check(case, out, q, cu, dtype, window, sinks, scale, hidden=None):
    got, qh = f64(out), f64(q)
    for b, n in enumerate(case.lens):
        x = qh[cu[b]:cu[b + 1]]
        ref, mag, lmag = paged.attend(x, case.k[b], case.v[b], n, window, sinks, scale,
                                      hidden[b] if hidden else ())
        vmax = np.abs(case.v[b]).max() if n else 0.0
        tol = tolerance(dtype, ref, mag, lmag, x, scale, vmax, n)
        err = np.abs(got[cu[b]:cu[b + 1]] - ref)
        assert (err <= tol).all(), (b, n, float((err / tol).max()), np.argwhere(err > tol)[:5])
        empty = ~mag.any(-1)
        assert not got[cu[b]:cu[b + 1]][empty].any()


def queries(case, counts, h_q, dtype, gain=1.0):
    cu = np.concatenate([[0], np.cumsum(counts)])
    return rounded(case.rng.normal(size=(cu[-1], h_q, case.d)) * gain, dtype), cu


CASES = [
    # lens, queries per sequence, h_kv, group, d, page, window, sinks
    ([1], [1], 1, 1, 64, 16, 0, 0),
    ([1], [1], 8, 4, 128, 16, 0, 0),
    ([17], [1], 2, 4, 128, 16, 0, 0),
    ([1000], [1], 2, 4, 128, 16, 0, 0),
    ([1025, 1, 0, 64, 333], [1] * 5, 2, 4, 128, 64, 0, 0),
    ([500, 129, 31], [1] * 3, 1, 8, 64, 32, 100, 4),
    ([300, 40], [1] * 2, 2, 5, 128, 16, 1, 0),
    ([300, 40], [1] * 2, 2, 3, 64, 128, 33, 50),     # sinks reach into the window of the short one
    ([260, 700], [1] * 2, 1, 16, 128, 256, 0, 0),    # more heads than one tile of rows
    ([77, 5, 200], [5] * 3, 2, 4, 64, 16, 0, 0),     # a few queries each
    ([77, 2, 200], [5] * 3, 1, 5, 128, 32, 20, 3),   # more queries than tokens: the first see nothing
    ([90, 64, 10, 0], [90, 1, 0, 3], 2, 4, 128, 16, 0, 0),  # prefill beside decode, none, and queries of an empty sequence
    ([300], [300], 1, 4, 128, 64, 0, 0),
    ([333, 129], [200, 129], 1, 4, 64, 16, 50, 4),
    ([400, 513], [400, 130], 1, 1, 128, 16, 128, 0),
    ([257], [129], 1, 3, 64, 32, 7, 300),            # sinks beyond the length
    ([200], [200], 1, 2, 128, 1024, 1, 1),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens,counts,h_kv,group,d,page,window,sinks", CASES)
def test_attend(dtype, lens, counts, h_kv, group, d, page, window, sinks):
    case = Case(len(lens) + lens[0], lens, h_kv, d, page)
    q, cu = queries(case, counts, h_kv * group, dtype)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = d ** -0.5
    out = case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu), window=window, sinks=sinks, bad=bad)
    check(case, out, q, cu, dtype, window, sinks, scale)
    if len(set(counts)) == 1:  # the same number of queries each: no cu_q needed
        same = case.cache.attend(q, i32(case.pages), i32(lens), window=window, sinks=sinks, bad=bad)
        assert torch.equal(out, same)
    assert bad.item() == 0


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("gain,spread,scale", [(20.0, 1.0, None), (1.0, 1e-5, None), (1e-3, 1e4, 0.3), (1.0, 1.0, -0.1),
                                               (1.0, 1.0, 0.0), (0.0, 1.0, None)])
def test_attend_magnitudes(nq, gain, spread, scale):
    """Peaked and flat softmax, tiny and huge values, negative and zero scale, zero queries."""
    case = Case(3, [400], 1, 128, 16, spread)
    q, cu = queries(case, [nq], 4, "fp16", gain)
    out = case.cache.attend(q, i32(case.pages), i32([400]), scale=scale)
    check(case, out, q, cu, "fp16", 0, 0, 128 ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("nq", [1, 3, 70])
@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 0), (50, 3)])
def test_visible_borders(nq, window, sinks):
    """Tokens next to every border of the mask hold values a thousand times the
    rest, so that one token seen or missed shows."""
    d, n, page = 64, 300, 16
    case = Case(9, [n], 1, d, page)
    q, cu = queries(case, [nq], 2, "fp16", 0.1)
    marks = {0, sinks - 1, sinks, n - 1, n - nq} | {p - window for p in range(n - nq, n)} | {p - window + 1 for p in range(n - nq, n)}
    marks = sorted(j for j in marks if 0 <= j < n)
    v = rounded(case.rng.choice([-1000.0, 1000.0], (len(marks), 1, d)), "fp16")
    slots = case.pages[0][np.array(marks) // page] * page + np.array(marks) % page
    case.cache.write(None, v, i32(slots))
    case.v[0] = case.v[0].copy()
    case.v[0][marks] = paged.stored(f64(v))
    out = case.cache.attend(q, i32(case.pages), i32([n]), window=window, sinks=sinks)
    check(case, out, q, cu, "fp16", window, sinks, d ** -0.5)


@pytest.mark.parametrize("nq", [1, 60])
def test_long_context(nq):
    case = Case(11, [9000, 4097], 1, 128, 64)
    q, cu = queries(case, [nq, nq], 4, "bf16", 2.0)
    out = case.cache.attend(q, i32(case.pages), i32(case.lens))
    rows = [0, nq - 1]
    got, qh = f64(out), f64(q)
    for b, n in enumerate(case.lens):
        for r in rows:  # the oracle on the first and the last query
            p = n - nq + r + 1
            x = qh[cu[b] + r:cu[b] + r + 1]
            ref, mag, lmag = paged.attend(x, case.k[b][:p], case.v[b][:p], p, 0, 0, 128 ** -0.5)
            tol = tolerance("bf16", ref, mag, lmag, x, 128 ** -0.5, np.abs(case.v[b]).max(), n)
            assert (np.abs(got[cu[b] + r] - ref[0]) <= tol[0]).all()


@pytest.mark.parametrize("counts", [[1, 1, 1], [4, 4, 4], [50, 2, 40]])
def test_bad_indices_are_not_followed(counts):
    """Page indices outside the pool hide their tokens, lengths are clamped to
    what the table holds, and both are reported."""
    lens, page = [100, 90, 80], 16
    case = Case(13, lens, 2, 64, page)
    q, cu = queries(case, counts, 4, "fp16")
    pages = case.pages.copy()
    pages[0, 2] = case.n_pages      # tokens 32..47
    pages[1, 0] = -7                # tokens 0..15
    pages[2, :] = 2 ** 31 - 1       # every token
    hidden = [set(range(32, 48)), set(range(16)), set(range(80))]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = case.cache.attend(q, i32(pages), i32(lens), cu_q=i32(cu), bad=bad)
    check(case, out, q, cu, "fp16", 0, 0, 64 ** -0.5, hidden)
    assert bad.item() > 0
    # entries that hold no visible token are not looked at
    bad.zero_()
    pages = case.pages.copy()
    pages[0, 0] = 999               # before the window of every query below
    out = case.cache.attend(q[:1], i32(pages[:1]), i32(lens[:1]), window=20, bad=bad)
    one = Case.__new__(Case)
    one.lens, one.k, one.v = lens[:1], case.k[:1], case.v[:1]
    check(one, out, q[:1], [0, 1], "fp16", 20, 0, 64 ** -0.5)
    assert bad.item() == 0
    # lengths beyond the table (clamped to it: its last page is hidden) and below zero, row offsets beyond the queries
    out = case.cache.attend(q, i32(case.pages), i32([-5, 10 ** 9, 80]), cu_q=i32([0, counts[0], cu[2], 10 ** 9]), bad=bad)
    assert bad.item() > 0 and not out[:counts[0]].any()
    good = case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu))
    assert torch.equal(out[cu[2]:], good[cu[2]:])
    out = case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32([cu[3], 0, -4, cu[3]]), bad=bad)
    torch.cuda.synchronize()


def test_rows_of_no_sequence_are_left():
    case = Case(15, [50, 60], 1, 128, 16)
    for counts in ([1, 1], [3, 2], [30, 20]):
        q, cu = queries(case, [7] + counts + [9], 4, "bf16")
        out = torch.full(q.shape, 7.25, dtype=q.dtype, device="cuda")
        case.cache.attend(q, i32(case.pages), i32(case.lens), cu_q=i32(cu[1:4]), out=out)
        assert (out[:7] == 7.25).all() and (out[cu[3]:] == 7.25).all()
        check(case, out, q, cu[1:], "bf16", 0, 0, 128 ** -0.5)


def test_spoilt_queries_spoil_their_own_rows_only():
    case = Case(17, [70, 90], 1, 128, 16)
    for counts in ([1, 1], [40, 40]):
        q, cu = queries(case, counts, 4, "fp16")
        good = case.cache.attend(q, i32(case.pages), i32(case.lens), cu_q=i32(cu))
        q2 = q.clone()
        q2[0, 1, 3], q2[-1, 2, 5] = float("nan"), float("inf")
        out = case.cache.attend(q2, i32(case.pages), i32(case.lens), cu_q=i32(cu))
        keep = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
        keep[0, 1] = keep[-1, 2] = False
        assert torch.equal(out[keep], good[keep])


def test_strided_queries_and_repeats():
    case = Case(19, [70, 90, 40], 2, 64, 16)
    wide = rounded(case.rng.normal(size=(3 * 9, (8 + 4) * 64)), "fp16")
    q = wide[:, 2 * 64:10 * 64].unflatten(1, (8, 64))
    cu = [0, 9, 18, 27]
    args = (i32(case.pages), i32(case.lens))
    a = case.cache.attend(q, *args)
    b = case.cache.attend(q.contiguous(), *args)
    assert torch.equal(a, b)
    check(case, a, q, cu, "fp16", 0, 0, 64 ** -0.5)
    # one page table for two sequences (a shared prefix)
    both = case.cache.attend(q[:2], i32(np.stack([case.pages[1]] * 2)), i32([90, 30]))
    assert torch.equal(both[0], case.cache.attend(q[:1], i32(case.pages[1:2]), i32([90]))[0])
    # results do not depend on the run
    for _ in range(3):
        assert torch.equal(case.cache.attend(q, *args), a)


# ---------------------------------------------------------------------------
# the three together


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_prefill_then_decode(window, sinks):
    """Prompts of different lengths written and attended to in chunks, then
    decoded token by token, against the oracle on the same tokens."""
    rng = np.random.default_rng(21)
    h_kv, group, d, page = 2, 4, 128, 16
    plan = [[33, 20, 1, 1, 1], [70, 0, 1, 1, 1], [5, 9, 1, 1, 1]]  # new tokens of each sequence per step
    totals = [sum(p) for p in plan]
    table = rng.permutation(3 * 8).reshape(3, 8)
    cache = PagedKVCache(24, page, h_kv, d)
    k = [rounded(tokens(rng, t, h_kv, d), "bf16") for t in totals]
    v = [rounded(rng.normal(size=(t, h_kv, d)), "bf16") for t in totals]
    q = [rounded(rng.normal(size=(t, h_kv * group, d)), "bf16") for t in totals]
    done = [0, 0, 0]
    for step in range(5):
        new = [p[step] for p in plan]
        pos = [np.arange(s, s + n) for s, n in zip(done, new)]
        slots = np.concatenate([table[b, p // page] * page + p % page for b, p in enumerate(pos)])
        pick = lambda xs: torch.cat([x[s:s + n] for x, s, n in zip(xs, done, new)])
        cache.write(pick(k), pick(v), i32(slots))
        done = [s + n for s, n in zip(done, new)]
        cu = np.concatenate([[0], np.cumsum(new)])
        out = cache.attend(pick(q), i32(table), i32(done), cu_q=i32(cu), window=window, sinks=sinks)
        one = Case.__new__(Case)
        one.lens = done
        one.k, one.v = ([paged.stored(f64(x[:s])) for x, s in zip(xs, done)] for xs in (k, v))
        check(one, out, pick(q), cu, "bf16", window, sinks, d ** -0.5)
    back, _ = cache.read(i32(table[1, np.arange(totals[1]) // page] * page + np.arange(totals[1]) % page), torch.float32)
    assert np.array_equal(f64(back).astype(np.float32), paged.stored(f64(k[1])).astype(np.float32))


@pytest.mark.parametrize("nq", [1, 50])
def test_streams_and_graphs(nq):
    """On a side stream; captured with the write before it and replayed with new
    inputs and lengths; two captured graphs with a workspace each in flight at once."""
    d, page, h_kv = 128, 16, 2
    case = Case(23, [100, 90], h_kv, d, page)
    q, cu = queries(case, [nq, nq], 8, "bf16")
    args = (i32(case.pages), i32(case.lens))
    want = case.cache.attend(q, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = case.cache.attend(q, *args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    bufs = []
    for i in range(2):
        lens = i32(case.lens)
        qq, out = q.clone(), torch.zeros_like(q)
        ws = torch.empty(max(16, case.cache.attend_workspace(2 * nq, 2, 8)), dtype=torch.uint8, device="cuda")
        kv = torch.zeros(2, h_kv, d, dtype=torch.bfloat16, device="cuda")
        slots = i32([-1, -1])
        case.cache.attend(qq, args[0], lens, out=out, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            case.cache.write(kv, kv, slots)
            case.cache.attend(qq, args[0], lens, out=out, ws=ws)
        bufs.append((g, qq, out, lens, kv, slots, ws))
    for rep in range(3):
        fresh = [rounded(case.rng.normal(size=q.shape), "bf16") for _ in range(2)]
        short = [[100 - rep, 77 + rep], [13 + rep, 90]]
        for (g, qq, out, lens, *_), x, n in zip(bufs, fresh, short):
            qq.copy_(x)
            lens.copy_(i32(n))
        streams = [torch.cuda.Stream() for _ in bufs]
        for s, (g, *_) in zip(streams, bufs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, out, *_), x, n in zip(bufs, fresh, short):
            assert torch.equal(out, case.cache.attend(x, args[0], i32(n)))
    # a replay that writes: the new token is the last one seen
    g, qq, out, lens, kv, slots, _ = bufs[0]
    x = rounded(case.rng.normal(size=(2, h_kv, d)), "bf16")
    kv.copy_(x)
    at = [99, 89]
    slots.copy_(i32([case.pages[b, at[b] // page] * page + at[b] % page for b in range(2)]))
    lens.copy_(i32(case.lens))
    qq.copy_(q)
    g.replay()
    for b in range(2):
        case.k[b][at[b]] = case.v[b][at[b]] = paged.stored(f64(x[b]))
    check(case, out, q, cu, "bf16", 0, 0, d ** -0.5)


def test_python_refusals():
    cache = PagedKVCache(4, 16, 2, 64)
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    s = i32([0, 1, 2])
    for call in (lambda: cache.write(k, k.bfloat16(), s), lambda: cache.write(k, k[:2], s), lambda: cache.write(k, k, s.long()),
                 lambda: cache.write(k, k, s[:2]), lambda: cache.write(k.double(), None, s), lambda: cache.write(None, None, s),
                 lambda: cache.write(k.cpu(), None, s), lambda: cache.write(k[:, :1], None, s), lambda: cache.write(k, k, s.cpu()),
                 lambda: cache.write(k.transpose(1, 2).contiguous().transpose(1, 2), None, s),
                 lambda: cache.read(s, torch.int32), lambda: cache.read(s, k=k.float()), lambda: cache.read(i32([0, 1, 2, 3])[::2]),
                 lambda: cache.attend(k.float(), i32([[0]]), i32([3])), lambda: cache.attend(k, i32([[0]]), i32([3]), window=-1),
                 lambda: cache.attend(k[:, :, :32], i32([[0]]), i32([3])), lambda: cache.attend(k, i32([[0], [1]]), i32([3])),
                 lambda: cache.attend(k, i32([[0]]), i32([3]), cu_q=i32([0, 1, 3])), lambda: cache.attend(k, i32([0]), i32([3])),
                 lambda: cache.attend(k, i32([[0]]), i32([3]), out=k.float()), lambda: cache.attend(k, i32([[0]]).long(), i32([3])),
                 lambda: cache.attend(k, i32([[0]]), i32([3]), scale=float("nan")),
                 lambda: PagedKVCache(4, 16, 2, 64, pool=torch.zeros(10, dtype=torch.uint8, device="cuda")),
                 lambda: PagedKVCache(4, 17, 2, 64)):
        with pytest.raises(abi.SFError):
            call()
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# sizes that reach every form of the kernels (fp64 reference on the device)


def reference(case, q, cu, b, row, window, sinks, scale):
    """One query row of sequence b in fp64 on the device: (out, sum p|v|, largest scale sum |q||k|) per head."""
    n = case.lens[b]
    x = q[cu[b] + row].double()
    p = n - (cu[b + 1] - cu[b]) + row
    j = torch.arange(max(p + 1, 0), device="cuda")
    if window:
        j = j[(j > p - window) | (j < sinks)]
    k, v = (torch.as_tensor(t[b]).cuda()[j].repeat_interleave(q.shape[1] // case.h_kv, 1) for t in (case.k, case.v))
    w = torch.softmax(torch.einsum("hd,jhd->hj", x, k) * scale, -1)
    lmag = abs(scale) * torch.einsum("hd,jhd->hj", x.abs(), k.abs()).amax(-1)
    return f64(torch.einsum("hj,jhd->hd", w, v)), f64(torch.einsum("hj,jhd->hd", w, v.abs())), f64(lmag)


def spot_check(case, out, q, cu, dtype, window, sinks, rows):
    scale = case.d ** -0.5
    got, qh = f64(out), f64(q)
    for b, r in rows:
        if case.lens[b] - (cu[b + 1] - cu[b]) + r < 0:
            assert not got[cu[b] + r].any()
            continue
        ref, mag, lmag = reference(case, q, cu, b, r, window, sinks, scale)
        tol = tolerance(dtype, ref, mag, lmag, qh[cu[b] + r], scale, np.abs(case.v[b]).max(), case.lens[b])
        err = np.abs(got[cu[b] + r] - ref)
        assert (err <= tol).all(), (b, r, float((err / tol).max()))


@pytest.mark.parametrize("batch,nq,h_kv,group,d,window", [
    (70, 1, 8, 4, 128, 0),     # more items than CTAs
    (30, 1, 8, 4, 64, 40),     # fewer items than CTAs: an entry each
    (50, 3, 4, 5, 128, 0),     # two columns of rows
    (40, 3, 2, 7, 64, 100),    # three
    (33, 8, 2, 8, 128, 0),     # two items per sequence
    (9, 40, 8, 4, 128, 0),     # many-row items, one tile and two
    (40, 100, 8, 4, 64, 64),   # more of them than CTAs
])
def test_batches(batch, nq, h_kv, group, d, window):
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 700, batch)]
    lens[3], lens[5] = 0, 1
    case = Case(batch, lens, h_kv, d, 32)
    q, cu = queries(case, [nq] * batch, h_kv * group, "bf16")
    out = case.cache.attend(q, i32(case.pages), i32(lens), window=window, sinks=3)
    again = case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu), window=window, sinks=3)
    assert torch.equal(out, again)
    rows = [(int(b), int(r)) for b, r in zip(rng.integers(0, batch, 40), rng.integers(0, nq, 40))] + [(3, 0), (5, nq - 1)]
    spot_check(case, out, q, cu, "bf16", window, 3, rows)


def test_workspace_sizes_kept():
    """A server's batches come in ever new shapes: what is kept of them is bounded."""
    cache = PagedKVCache(1, 16, 1, 64)
    sizes = [cache.attend_workspace(n, 1, 4) for n in range(1, 2500)]
    assert len(cache._ws_bytes) <= 1024
    assert sizes == [cache.attend_workspace(n, 1, 4) for n in range(1, 2500)]


@pytest.mark.parametrize("h_kv,group,d", [(1, 64, 128), (1, 65, 64), (2, 80, 128), (1, 300, 64)])
def test_many_heads_per_kv_head(h_kv, group, d):
    """One query per sequence whose heads alone fill the few-row kernel or go
    to the many-row one, up to more than one of its tiles."""
    lens = [300, 0, 1, 2049]
    case = Case(group, lens, h_kv, d, 16)
    q, cu = queries(case, [1] * 4, h_kv * group, "bf16")
    out = case.cache.attend(q, i32(case.pages), i32(lens), window=200, sinks=2)
    check(case, out, q, cu, "bf16", 200, 2, d ** -0.5)
    assert torch.equal(out, case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu), window=200, sinks=2))


@pytest.mark.parametrize("d", [64, 128])
def test_mixed_long_batch(d):
    """Chunks of thousands of queries, drafts and single tokens in one call; the
    bounded waits of the kernels all end by themselves."""
    lens, counts = [3000, 5000, 1, 2500, 700, 4096], [3000, 1000, 1, 1, 7, 4096]
    case = Case(31, lens, 2, d, 64)
    q, cu = queries(case, counts, 8, "fp16")
    left, n = ctypes.c_uint(), 0
    abi.sf_device_wait_timeouts(ctypes.byref(left), 1)
    for window, sinks in ((0, 0), (1000, 4)):
        for _ in range(10):
            out = case.cache.attend(q, i32(case.pages), i32(lens), cu_q=i32(cu), window=window, sinks=sinks)
        rows = [(b, int(r)) for b in range(6) for r in case.rng.integers(0, counts[b], 8)]
        spot_check(case, out, q, cu, "fp16", window, sinks, rows)
    abi.check(abi.sf_device_wait_timeouts(ctypes.byref(left), 0), "sf_device_wait_timeouts")


def test_offsets_past_32_bits():
    """A pool of 5 GB whose last pages are used."""
    page, h_kv, d = 64, 8, 128
    n_pages = 5 * 10 ** 9 // (page * h_kv * 160)
    cache = PagedKVCache(n_pages, page, h_kv, d)
    rng = np.random.default_rng(0)
    k, v = rounded(tokens(rng, 200, h_kv, d), "bf16"), rounded(rng.normal(size=(200, h_kv, d)), "bf16")
    table = np.array([[n_pages - 1, 0, n_pages - 3, n_pages // 2]])
    slots = table[0, np.arange(200) // page] * page + np.arange(200) % page
    cache.write(k, v, i32(slots))
    kk, vv = cache.read(i32(slots), torch.float32)
    assert np.array_equal(f64(kk).astype(np.float32), paged.stored(f64(k)).astype(np.float32))
    case = Case.__new__(Case)
    case.lens, case.h_kv, case.d, case.rng = [200], h_kv, d, rng
    case.k, case.v = [paged.stored(f64(k))], [paged.stored(f64(v))]
    for nq in (1, 100):
        q, cu = queries(case, [nq], 32, "bf16")
        out = cache.attend(q, i32(table), i32([200]))
        spot_check(case, out, q, cu, "bf16", 0, 0, [(0, 0), (0, nq - 1)])


def test_wide_window_is_no_window():
    """Windows up to the largest int behave as none; sinks likewise as all."""
    case = Case(33, [300], 1, 64, 16)
    for nq in (1, 100):
        q, _ = queries(case, [nq], 4, "fp16")
        args = (q, i32(case.pages), i32([300]))
        full = case.cache.attend(*args)
        for window, sinks in ((300, 0), (2 ** 31 - 1, 5), (1, 2 ** 31 - 1), (7, 300)):
            assert torch.equal(case.cache.attend(*args, window=window, sinks=sinks), full), (window, sinks)
