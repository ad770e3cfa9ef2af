"""Which stream the memory of a call belongs to, on the host: the launches, the
allocator and the streams are stand-ins that note who asked for what."""
import contextlib

import pytest
import torch

from bit_decode_selective_b200 import abi, ops

CPU = torch.device("cpu")
I32 = dict(dtype=torch.int32)


class Memory:
    """An allocation: the stream it belongs to and the streams it waits for before it is used again."""

    def __init__(self, shape, dtype, owner):
        self.shape = (shape,) if isinstance(shape, int) else torch.Size(shape)
        self.dtype, self.owner, self.device = dtype, owner, CPU
        self.recorded = []

    def data_ptr(self):
        return id(self)

    def numel(self):
        return self.nbytes

    nbytes = 1 << 30

    def record_stream(self, stream):
        self.recorded.append(stream)


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, CPU


class Streams:
    """The current stream and everything that was allocated, in order."""

    def __init__(self, monkeypatch):
        self.main, self.side = (FakeStream(h) for h in (0, 7))
        self.now, self.memory, self.launches, self.recorded = self.main, [], [], []
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, stream: self.recorded.append((id(t), stream)))
        monkeypatch.setattr(torch.cuda, "stream", self.on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(ops, "_current_stream", lambda index: self.now.cuda_stream)

    @contextlib.contextmanager
    def on(self, stream):
        before, self.now = self.now, stream if stream is not None else self.now
        yield
        self.now = before

    def new_empty(self, shape, dtype=torch.uint8):
        self.memory.append(Memory(shape, dtype, self.now))
        return self.memory[-1]

    def launch(self, *args):
        self.launches.append(args[-1])
        return 0


@pytest.fixture
def streams(monkeypatch):
    return Streams(monkeypatch)


def paged_cache(streams):
    cache = ops.PagedKVCache.__new__(ops.PagedKVCache)
    cache.n_pages, cache.page, cache.h_kv, cache.d = 4, 16, 2, 64
    cache.device, cache._index_of_device, cache._ref = CPU, 0, None
    cache.pool = Memory((1,), torch.uint8, streams.main)
    cache.pool.new_empty = streams.new_empty
    cache._ws_bytes = {(3, 1, 2): 4096}
    cache._fn = {name: streams.launch for name in ("sf_kvp_write", "sf_kvp_read", "sf_kvp_attend")}
    return cache


def test_paged_calls_allocate_on_the_stream_that_writes(streams):
    cache = paged_cache(streams)
    q = torch.zeros(3, 2, 64, dtype=torch.float16)
    pages, lens, slots = torch.zeros(1, 1, **I32), torch.zeros(1, **I32), torch.zeros(3, **I32)
    cache.attend(q, pages, lens, stream=streams.side)
    out, ws = streams.memory
    assert out.owner is streams.side and ws.owner is streams.side
    assert streams.main in out.recorded  # the caller's stream may still use it when it is dropped
    cache.read(slots, stream=streams.side)
    for t in streams.memory[2:]:
        assert t.owner is streams.side and streams.main in t.recorded
    assert len(streams.memory) == 4 and streams.launches == [7, 7] and streams.now is streams.main


def test_paged_calls_keep_what_they_are_given(streams):
    """Tensors given to a call on another stream are kept until its work is done; on
    the current stream nothing needs keeping."""
    cache = paged_cache(streams)
    k, v, q = (torch.zeros(3, 2, 64, dtype=torch.float16) for _ in range(3))
    pages, lens, cu, bad, slots = (torch.zeros(s, **I32) for s in ((1, 1), 1, 2, 1, 3))
    out, ws, kk, vv = torch.zeros_like(q), torch.zeros(4096, dtype=torch.uint8), torch.zeros_like(k), torch.zeros_like(v)
    calls = {
        lambda s: cache.write(k, v, slots, bad=bad, stream=s): (k, v, slots, bad),
        lambda s: cache.read(slots, k=kk, v=vv, bad=bad, stream=s): (slots, kk, vv, bad),
        lambda s: cache.attend(q, pages, lens, cu_q=cu, out=out, bad=bad, ws=ws, stream=s): (q, pages, lens, cu, out, bad, ws),
    }
    for call, given in calls.items():
        streams.recorded.clear(), cache.pool.recorded.clear()
        call(None)
        assert not streams.recorded and not cache.pool.recorded
        call(streams.side)
        assert {(id(t), streams.side) for t in given} <= set(streams.recorded)
        assert cache.pool.recorded == [streams.side]
    assert not streams.memory


class Half(Memory):
    """An fp16 input on the current stream."""

    is_cuda = True

    def __init__(self, streams, *shape, dtype=torch.float16):
        super().__init__(shape, dtype, streams.main)
        self.new_empty = streams.new_empty

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True


def weights():
    w = ops.QuantWeights.__new__(ops.QuantWeights)
    w.n, w.k, w.b, w.r, w.group, w.desc = 64, 2048, 2, 2, 128, abi.sf_wq()
    return w


def kv_cache():
    c = ops.KVCache.__new__(ops.KVCache)
    c.batch, c.h_kv, c.t_max, c.d, c.desc = 1, 2, 1024, 128, abi.sf_kv()
    return c


# call, what it allocates and hands out, its workspaces
@pytest.mark.parametrize("call,returned,spaces", [
    (lambda s, at: weights().gemv(Half(s, 1, 2048), stream=at), 2, 1),
    (lambda s, at: weights().gemv_split(Half(s, 1, 2048), None, stream=at), 2, 0),
    (lambda s, at: weights().fit_refinements(Half(s, 64, 2048, dtype=torch.float32), Half(s, 8, 2048), want_delta=True,
                                             stream=at), 1, 1),
    (lambda s, at: ops.select_channels(Half(s, 1, 2048), stream=at), 1, 0),
    (lambda s, at: kv_cache().score_select(Half(s, 1, 8, 128), 100, 4, want_scores=True, stream=at), 3, 1),
    (lambda s, at: kv_cache().logits_fma(Half(s, 1, 8, 128), 100, stream=at), 1, 1),
    (lambda s, at: kv_cache().attn_refined(Half(s, 1, 8, 128), 100, None, 4, stream=at), 1, 1),
    (lambda s, at: kv_cache().attend_selective(Half(s, 1, 8, 128), 100, 4, stream=at), 2, 1),
], ids=["gemv", "gemv_split", "fit", "select", "score_select", "logits_fma", "attn_refined", "attend_selective"])
def test_nested_calls_allocate_on_the_stream_that_writes(streams, monkeypatch, call, returned, spaces):
    for name in vars(abi):
        if name.startswith("sf_") and not isinstance(getattr(abi, name), type):
            monkeypatch.setattr(abi, name, lambda *args: 256)
    monkeypatch.setattr(ops, "check", lambda status, where: None)
    call(streams, streams.side)
    assert len(streams.memory) == returned + spaces
    assert all(t.owner is streams.side for t in streams.memory)
    assert sum(t.recorded == [streams.main] for t in streams.memory) == returned
    streams.memory.clear()
    call(streams, None)
    assert all(t.owner is streams.main and not t.recorded for t in streams.memory)
