"""Torch-facing helpers over the C ABI: they allocate caller-owned buffers with
PyTorch (device memory and streams are all PyTorch is used for) and pass raw
pointers to the CUDA library.  No arithmetic of the method happens here."""
from __future__ import annotations

import ctypes

import torch

from . import abi
from .abi import check


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _empty(like, shape, dtype, stream, returned=True):
    """A new tensor on `like`'s device that work on `stream` (None: the current one)
    writes first.  It belongs to that stream: memory that the current stream has
    given back may still be in use by work queued there, which `stream` does not
    wait for.  `returned`: the caller gets it, so once dropped it is not used again
    before the work that the current stream holds by then."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    if returned:
        t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _used_on(stream, *tensors):
    """The memory of `tensors` (None: not given) is not used again before the work
    that `stream` holds when they are dropped."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _f16(t: torch.Tensor) -> torch.Tensor:
    assert t.dtype in (torch.float16, torch.int16, torch.uint16), t.dtype
    assert t.is_cuda and t.is_contiguous()
    return t


class QuantWeights:
    """A nested-quantised weight matrix W[n][k] (format: include/sf.h, sf_wq)."""

    def __init__(self, n: int, k: int, b: int, r: int, group: int = 128, device="cuda",
                 with_refine: bool = True):
        sizes = [ctypes.c_size_t() for _ in range(3)]
        check(abi.sf_wq_bytes(n, k, b, r, group, *[ctypes.byref(s) for s in sizes]), "sf_wq_bytes")
        self.n, self.k, self.b, self.r, self.group = n, k, b, r, group
        self.base = torch.empty(sizes[0].value, dtype=torch.uint8, device=device)
        self.refine = torch.empty(sizes[1].value, dtype=torch.uint8, device=device) if with_refine else None
        self.sz = torch.empty(sizes[2].value // 2, dtype=torch.int16, device=device)
        self.desc = abi.sf_wq(n, k, b, r, group, self.base.data_ptr(),
                              self.refine.data_ptr() if with_refine else None, self.sz.data_ptr())

    @classmethod
    def pack(cls, w: torch.Tensor, b: int, r: int, group: int = 128) -> "QuantWeights":
        assert w.dtype == torch.float32 and w.is_cuda and w.is_contiguous() and w.dim() == 2
        q = cls(w.shape[0], w.shape[1], b, r, group, device=w.device)
        check(abi.sf_pack_nested(_p(w), ctypes.byref(q.desc), _stream()), "sf_pack_nested")
        return q

    def fit_refinements(self, w: torch.Tensor, x_cal: torch.Tensor, chunk: int = 1024, kch: int = 32,
                        alpha: float = 0.01, want_delta: bool = False, stream=None):
        """Refit the refinement codes on calibration activations x_cal [n_cal][k]
        (sf_fit_refinements); w is the fp32 matrix this one was packed from.
        Returns the fitted corrections [n][k] fp64 when want_delta."""
        assert w.dtype == torch.float32 and w.is_contiguous() and tuple(w.shape) == (self.n, self.k)
        x_cal = _f16(x_cal)
        n_cal = x_cal.shape[0]
        nbytes = abi.sf_fit_refinements_workspace_bytes(self.n, self.k, n_cal, chunk, kch)
        ws = _empty(w, nbytes, torch.uint8, stream, returned=False)
        delta = _empty(w, (self.n, self.k), torch.float64, stream) if want_delta else None
        check(abi.sf_fit_refinements(_p(w), ctypes.byref(self.desc), _p(x_cal), n_cal, chunk, kch, alpha, _p(delta),
                                     _p(ws), nbytes, _stream(stream)), "sf_fit_refinements")
        return delta

    def refine_rows(self) -> torch.Tensor:
        """The refinement buffer viewed as [k][n*r/8] rows (one per input channel)."""
        return self.refine.view(self.k, self.n * self.r // 8)

    def unpack(self):
        qb = torch.empty((self.n, self.k), dtype=torch.uint8, device=self.base.device)
        rho = torch.empty_like(qb) if self.refine is not None else None
        check(abi.sf_unpack_codes(ctypes.byref(self.desc), _p(qb), _p(rho), _stream()), "sf_unpack_codes")
        return qb, rho

    def gemv(self, x: torch.Tensor, chunk: int = 1024, kch: int = 32, sel_in=None,
             refine_rows=None, y=None, sel_out=None, ws=None, stream=None):
        """y = W~ x (sf_gemv_refined).  Returns (y [batch][n] fp32, selection)."""
        x = _f16(x if x.dim() == 2 else x.view(1, -1))
        batch = x.shape[0]
        if y is None:
            y = _empty(x, (batch, self.n), torch.float32, stream)
        if kch > 0 and sel_in is None and sel_out is None:
            sel_out = _empty(x, (batch, self.k // chunk, kch), torch.int32, stream)
        if ws is None:
            need = abi.sf_gemv_workspace_bytes(ctypes.byref(self.desc), batch, chunk, kch)
            ws = _empty(x, max(need, 16), torch.uint8, stream, returned=False)
        check(abi.sf_gemv_refined(ctypes.byref(self.desc), _p(x), batch, chunk, kch, _p(sel_in),
                                  _p(sel_out), _p(refine_rows), _p(y), _p(ws), ws.numel(), _stream(stream)),
              "sf_gemv_refined")
        return y, (sel_in if sel_in is not None else sel_out)

    def correction(self, x: torch.Tensor, sel, y, chunk: int = 1024, kch: int = 32,
                   refine_rows=None, stream=None):
        """y += (W~ - W^) x over the selected channels (sf_gemv_correction)."""
        x = _f16(x if x.dim() == 2 else x.view(1, -1))
        check(abi.sf_gemv_correction(ctypes.byref(self.desc), _p(x), x.shape[0], chunk, kch, _p(sel),
                                     _p(refine_rows), _p(y), _stream(stream)),
              "sf_gemv_correction")
        return y


    def gemv_split(self, x: torch.Tensor, sel, chunk: int = 1024, kch: int = 32, refine_rows=None,
                   y_base=None, y_corr=None, stream=None):
        """Base product and correction to separate outputs (sf_gemv_refined_split).
        Returns (y_base, y_corr), each [batch][n] fp32."""
        x = _f16(x if x.dim() == 2 else x.view(1, -1))
        batch = x.shape[0]
        if y_base is None:
            y_base = _empty(x, (batch, self.n), torch.float32, stream)
        if y_corr is None:
            y_corr = _empty(x, (batch, self.n), torch.float32, stream)
        check(abi.sf_gemv_refined_split(ctypes.byref(self.desc), _p(x), batch, chunk, kch, _p(sel),
                                        _p(refine_rows), _p(y_base), _p(y_corr), _stream(stream)),
              "sf_gemv_refined_split")
        return y_base, y_corr


def select_channels(x: torch.Tensor, chunk: int = 1024, kch: int = 32, sel=None, stream=None):
    x = _f16(x if x.dim() == 2 else x.view(1, -1))
    batch, k = x.shape
    if sel is None:
        sel = _empty(x, (batch, k // chunk, kch), torch.int32, stream)
    check(abi.sf_select_channels(_p(x), batch, k, chunk, kch, _p(sel), _stream(stream)),
          "sf_select_channels")
    return sel


class KVCache:
    """`batch` nested-quantised KV caches (format: include/sf.h, sf_kv)."""

    def __init__(self, batch: int, h_kv: int, t_max: int, b: int = 2, r: int = 2, d: int = 128,
                 group: int = 32, device="cuda"):
        sizes = [ctypes.c_size_t() for _ in range(3)]
        check(abi.sf_kv_bytes(batch, h_kv, d, t_max, b, r, group, *[ctypes.byref(s) for s in sizes]),
              "sf_kv_bytes")
        mk = lambda nbytes: torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.batch, self.h_kv, self.t_max, self.b, self.r, self.d, self.group = batch, h_kv, t_max, b, r, d, group
        self.kb, self.kr, self.vb, self.vr = mk(sizes[0].value), mk(sizes[1].value), mk(sizes[0].value), mk(sizes[1].value)
        self.ksz = torch.zeros(sizes[2].value // 2, dtype=torch.int16, device=device)
        self.vsz = torch.zeros(sizes[2].value // 2, dtype=torch.int16, device=device)
        self.desc = abi.sf_kv(batch, h_kv, d, t_max, b, r, group, self.kb.data_ptr(), self.kr.data_ptr(),
                              self.vb.data_ptr(), self.vr.data_ptr(), self.ksz.data_ptr(), self.vsz.data_ptr())

    def pack_tokens(self, k, v, t0: int, stream=None):
        """k, v: [batch][h_kv][nt][d] fp16 (either may be None)."""
        nt = (k if k is not None else v).shape[2]
        check(abi.sf_kv_pack_tokens(ctypes.byref(self.desc), _p(k), _p(v), t0, nt, _stream(stream)),
              "sf_kv_pack_tokens")

    def unpack(self, which: int, t: int):
        dev = self.kb.device
        qb = torch.empty((self.batch, self.h_kv, t, self.d), dtype=torch.uint8, device=dev)
        rho = torch.empty_like(qb)
        check(abi.sf_kv_unpack_codes(ctypes.byref(self.desc), which, t, _p(qb), _p(rho), _stream()),
              "sf_kv_unpack_codes")
        return qb, rho

    def score_select_workspace(self, t: int, h_q: int, k_tok: int, logits_given: bool) -> int:
        return abi.sf_kv_score_select_workspace_bytes(ctypes.byref(self.desc), t, h_q, k_tok,
                                                      int(logits_given))

    def score_select(self, q: torch.Tensor, t: int, k_tok: int, logits=None, scores=None,
                     want_logits: bool = True, want_scores: bool = False, sel=None, ws=None,
                     stream=None):
        q = _f16(q)
        h_q = q.shape[1]
        if logits is None and want_logits:
            logits = _empty(q, (self.batch, h_q, t), torch.float32, stream)
        if scores is None and want_scores:
            scores = _empty(q, (self.batch, self.h_kv, t), torch.float32, stream)
        if sel is None:
            sel = _empty(q, (self.batch, self.h_kv, k_tok), torch.int32, stream)
        need = self.score_select_workspace(t, h_q, k_tok, logits is not None)
        if ws is None:
            ws = _empty(q, max(need, 16), torch.uint8, stream, returned=False)
        check(abi.sf_kv_score_select(ctypes.byref(self.desc), t, _p(q), h_q, k_tok, _p(sel), _p(logits),
                                     _p(scores), _p(ws), ws.numel(), _stream(stream)),
              "sf_kv_score_select")
        return sel, logits, scores

    def logits_fma(self, q: torch.Tensor, t: int, logits=None, ws=None, stream=None):
        """The base logits on the CUDA cores (sf_kv_logits_fma): [batch][h_q][t] fp32."""
        q = _f16(q)
        h_q = q.shape[1]
        if logits is None:
            logits = _empty(q, (self.batch, h_q, t), torch.float32, stream)
        need = abi.sf_kv_logits_fma_workspace_bytes(ctypes.byref(self.desc), t, h_q)
        if ws is None:
            ws = _empty(q, max(need, 16), torch.uint8, stream, returned=False)
        check(abi.sf_kv_logits_fma(ctypes.byref(self.desc), t, _p(q), h_q, _p(logits), _p(ws), ws.numel(),
                                   _stream(stream)), "sf_kv_logits_fma")
        return logits

    def attn_workspace(self, t: int, h_q: int, k_tok: int, n_splits: int = 0) -> int:
        return abi.sf_kv_attn_workspace_bytes(ctypes.byref(self.desc), t, h_q, k_tok, n_splits)

    def attn_refined(self, q: torch.Tensor, t: int, sel, k_tok: int, n_splits: int = 0, out=None,
                     ws=None, stream=None):
        q = _f16(q)
        h_q = q.shape[1]
        if out is None:
            out = _empty(q, (self.batch, h_q, self.d), torch.float32, stream)
        need = self.attn_workspace(t, h_q, k_tok, n_splits)
        if ws is None:
            ws = _empty(q, max(need, 16), torch.uint8, stream, returned=False)
        check(abi.sf_kv_attn_refined(ctypes.byref(self.desc), t, _p(q), h_q, _p(sel), k_tok, n_splits,
                                     _p(out), _p(ws), ws.numel(), _stream(stream)),
              "sf_kv_attn_refined")
        return out

    def attend_workspace(self, t: int, h_q: int, k_tok: int, logits_given: bool) -> int:
        return abi.sf_kv_attend_selective_workspace_bytes(ctypes.byref(self.desc), t, h_q, k_tok,
                                                          int(logits_given))

    def attend_selective(self, q: torch.Tensor, t: int, k_tok: int, sel=None, logits=None,
                         out=None, ws=None, stream=None):
        """Score, select and attend in one call.  Returns (out, sel)."""
        q = _f16(q)
        h_q = q.shape[1]
        if out is None:
            out = _empty(q, (self.batch, h_q, self.d), torch.float32, stream)
        if sel is None:
            sel = _empty(q, (self.batch, self.h_kv, k_tok), torch.int32, stream)
        need = self.attend_workspace(t, h_q, k_tok, logits is not None)
        if ws is None:
            ws = _empty(q, max(need, 16), torch.uint8, stream, returned=False)
        check(abi.sf_kv_attend_selective(ctypes.byref(self.desc), t, _p(q), h_q, k_tok, _p(sel),
                                         _p(logits), _p(out), _p(ws), ws.numel(), _stream(stream)),
              "sf_kv_attend_selective")
        return out, sel


_DTYPES = {torch.float16: abi.SF_F16, torch.bfloat16: abi.SF_BF16, torch.float32: abi.SF_F32}

# The handle of a device's current stream, without a Stream object around it
# (2 us less per call; single-token calls take a few).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _refuse(where: str, message: str):
    return abi.SFError(abi.SF_ERR_INVALID_ARG, where, message)


class PagedKVCache:
    """A pool of `n_pages` pages of `page` tokens, each token and KV head held as
    4-bit codes with fp16 grids over 32 elements (format: include/sf.h, sf_kvp).
    Sequences of any length share it through page tables; the slot of a token is
    page_index * page + place in the page.  `pool`: an existing buffer of that
    format instead of a new one.

    Calls with `stream` run there, and the caller orders that stream behind the
    work that fills their arguments and before the work that uses their results.
    Memory that a call allocates itself needs no such order, and tensors given to
    one may be dropped as soon as it returns."""

    def __init__(self, n_pages: int, page: int, h_kv: int, d: int = 128, device="cuda", pool=None):
        size = ctypes.c_size_t()
        check(abi.sf_kvp_bytes(n_pages, page, h_kv, d, ctypes.byref(size)), "sf_kvp_bytes")
        if pool is None:
            pool = torch.zeros(size.value, dtype=torch.uint8, device=device)
        if not (pool.is_cuda and pool.dtype == torch.uint8 and pool.is_contiguous() and pool.numel() == size.value):
            raise _refuse("PagedKVCache", f"pool must be {size.value} contiguous uint8 on a CUDA device")
        self.n_pages, self.page, self.h_kv, self.d, self.pool = n_pages, page, h_kv, d, pool
        self.device = pool.device
        self.desc = abi.sf_kvp(n_pages, page, h_kv, d, pool.data_ptr())
        self._ref = ctypes.byref(self.desc)
        self._ws_bytes = {}
        self._index_of_device = self.device.index
        self._fn = {name: getattr(abi.lib(), name) for name in ("sf_kvp_write", "sf_kvp_read", "sf_kvp_attend")}

    def _run(self, where, stream, *args):
        """The entry point on `stream` (default: the current one) of the cache's device."""
        index = self._index_of_device
        s = _current_stream(index) if stream is None else stream.cuda_stream
        if torch.cuda.current_device() == index:
            status = self._fn[where](self._ref, *args, s)
        else:
            with torch.cuda.device(index):
                status = self._fn[where](self._ref, *args, s)
        if status:
            check(status, where)

    def _index(self, t, where, name, *shape):
        if t.dtype != torch.int32 or t.device != self.device or t.shape != shape or not t.is_contiguous():
            raise _refuse(where, f"{name} must be contiguous int32 of shape {shape} on {self.device}")
        return t.data_ptr()

    def _rows(self, t, where, name, heads):
        """Pointer, row and head strides of [n][heads][d] rows with unit stride inside a head."""
        shape, stride = t.shape, t.stride()
        if (len(shape) != 3 or shape[1] != heads or shape[2] != self.d or t.device != self.device
                or (stride[2] != 1 and shape[0])):
            raise _refuse(where, f"{name} must be [n][{heads}][{self.d}] on {self.device}, elements of a head consecutive")
        return t.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if heads > 1 else 0

    def _bad(self, bad, where):
        if bad is None:
            return None
        if bad.dtype != torch.int32 or bad.device != self.device or bad.numel() != 1:
            raise _refuse(where, "bad must be one int32 on the cache's device")
        return bad.data_ptr()

    def write(self, k, v, slots, bad=None, stream=None):
        """Quantise tokens k, v [n][h_kv][d] (fp16, bf16 or fp32; either may be
        None) into `slots` [n] int32 (sf_kvp_write); -1 skips a token.  `bad`
        (one int32) counts slots outside the pool."""
        where = "sf_kvp_write"
        some = k if k is not None else v
        if some is None or some.dtype not in _DTYPES or some.dim() != 3:
            raise _refuse(where, "k or v must be given, [n][h_kv][d] of fp16, bf16 or fp32")
        n = some.shape[0]
        if v is not None and (v.dtype != some.dtype or v.shape[0] != n):
            raise _refuse(where, "k and v must be of one type and number of tokens")
        kp, kr, kh = self._rows(k, where, "k", self.h_kv) if k is not None else (None, 0, 0)
        vp, vr, vh = self._rows(v, where, "v", self.h_kv) if v is not None else (None, 0, 0)
        self._run(where, stream, kp, kr, kh, vp, vr, vh, _DTYPES[some.dtype], n,
                  self._index(slots, where, "slots", n), self._bad(bad, where))
        _used_on(stream, k, v, slots, bad, self.pool)

    def read(self, slots, dtype=torch.float16, k=None, v=None, bad=None, stream=None):
        """The values of `slots` [n] int32: (k, v), each [n][h_kv][d] of `dtype`
        (sf_kvp_read).  Rows of -1 and of slots outside the pool are zeros."""
        where = "sf_kvp_read"
        if dtype not in _DTYPES:
            raise _refuse(where, "dtype must be fp16, bf16 or fp32")
        n = slots.numel()
        shape = (n, self.h_kv, self.d)
        k = self._out(k, where, "k", shape, dtype, stream)
        v = torch.empty_like(k) if v is None and stream is None else self._out(v, where, "v", shape, dtype, stream)
        self._run(where, stream, self._index(slots, where, "slots", n), n, k.data_ptr(), v.data_ptr(), _DTYPES[dtype],
                  self._bad(bad, where))
        _used_on(stream, slots, k, v, bad, self.pool)
        return k, v

    def _out(self, t, where, name, shape, dtype, stream):
        """An output of the given shape: `t` where it is given, else a new tensor."""
        if t is None:
            return _empty(self.pool, shape, dtype, stream)
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != self.device:
            raise _refuse(where, f"{name} must be contiguous {dtype} of shape {tuple(shape)} on {self.device}")
        return t

    def attend_workspace(self, n_q: int, batch: int, h_q: int) -> int:
        key = (n_q, batch, h_q)
        need = self._ws_bytes.get(key)
        if need is None:
            with torch.cuda.device(self.device):
                need = abi.sf_kvp_attend_workspace_bytes(self._ref, n_q, batch, h_q)
            if len(self._ws_bytes) >= 1024:  # ragged batches come in endless shapes
                self._ws_bytes.clear()
            self._ws_bytes[key] = need
        return need

    def attend(self, q, pages, lens, cu_q=None, scale=None, window: int = 0, sinks: int = 0, out=None, bad=None,
               ws=None, stream=None):
        """Attention of queries q [n_q][h_q][d] (fp16 or bf16) over their
        sequences' cached tokens (sf_kvp_attend): pages [batch][max_pages] and
        lens [batch] int32; cu_q [batch + 1] int32 where the sequences have
        different numbers of queries; scale defaults to d ** -0.5.  A query sees
        the tokens up to its own, with window > 0 only the last `window` of them
        and the first `sinks`.  Returns out [n_q][h_q][d]."""
        where = "sf_kvp_attend"
        if q.dim() != 3 or q.dtype not in _DTYPES:
            raise _refuse(where, "q must be [n_q][h_q][d], fp16 or bf16")
        if lens.dim() != 1 or pages.dim() != 2:
            raise _refuse(where, "lens must be [batch], pages [batch][max_pages]")
        n_q, h_q, _ = q.shape
        batch, max_pages = pages.shape
        qp, qr, qh = self._rows(q, where, "q", h_q)
        if out is None and stream is None and q.is_contiguous():
            out = torch.empty_like(q)
        else:
            out = self._out(out, where, "out", q.shape, q.dtype, stream)
        if ws is None:
            ws = _empty(self.pool, self.attend_workspace(n_q, batch, h_q), torch.uint8, stream, returned=False)
        elif ws.device != self.device or not ws.is_contiguous():
            raise _refuse(where, "ws must be contiguous, on the cache's device")
        self._run(where, stream, qp, qr, qh, _DTYPES[q.dtype], n_q,
                  None if cu_q is None else self._index(cu_q, where, "cu_q", batch + 1),
                  self._index(pages, where, "pages", batch, max_pages), max_pages,
                  self._index(lens, where, "lens", batch), batch, h_q, self.d ** -0.5 if scale is None else scale,
                  window, sinks, out.data_ptr(), self._bad(bad, where), ws.data_ptr(), ws.nbytes)
        _used_on(stream, q, pages, lens, cu_q, out, bad, ws, self.pool)
        return out
