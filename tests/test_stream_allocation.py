"""A call that is given a stream makes what it allocates on that stream (memory of the current one may
still be written by kernels pending there, and is handed on there when the call drops it), and
tells the allocator that its results are read on the current stream.  Without a GPU: the library is
a stand-in that launches nothing, and the allocations are recorded."""
import contextlib
import types

import pytest
import torch

import mla_absorbed_latent_mtp_b200 as m

S = object()  # the stream
B, Q, L, P = 2, 3, 130, 5


class FakeLib:
    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith("workspace_bytes") else 0


class Record:
    def __init__(self, monkeypatch):
        self.inside, self.made, self.outside, self.read = False, [], [], []
        m._get_torch()
        for name in ("empty", "zeros"):
            monkeypatch.setattr(torch, name, self.allocator(getattr(torch, name)))
        monkeypatch.setattr(m, "_lib", FakeLib())
        monkeypatch.setattr(m, "_check_cuda", lambda *t: 0)
        monkeypatch.setattr(m, "_check_current", lambda *t: None)
        monkeypatch.setattr(m, "_stream", lambda s: 0)
        monkeypatch.setattr(m, "_on", self.on)

    def allocator(self, make):
        def wrapped(*shape, **kw):
            kw.pop("device", None)
            t = make(*shape, **kw)
            (self.made if self.inside else self.outside).append(t)  # kept, so that ids stay theirs
            return t
        return wrapped

    def on(self, stream, call, *args):
        assert stream is S and not self.inside
        self.inside = True
        out = call(*args)
        self.inside = False
        self.read += [id(t) for t in (out if isinstance(out, tuple) else (out,))]
        return out


def bf(*shape):
    return torch.full(shape, 0, dtype=torch.bfloat16)


def i32(*shape):
    return torch.full(shape, 0, dtype=torch.int32)


def u8(*shape):
    return torch.full(shape, 0, dtype=torch.uint8)


QT, QH, W, CACHE, LENS = bf(B, Q, 64, 512), bf(B, Q, 64, 256), bf(64, 256, 512), bf(B, L, 512), i32(B)
POOL, TABLE, PACKED, INDICES, REFS = bf(P, 64, 512), i32(B, 3), u8(P, 64, 288), i32(B, Q, 16), i32(P)
CALLS = {
    "absorb_q": lambda: m.mla_absorb_q(QH, W, stream=S),
    "up_proj": lambda: m.mla_up_proj(QT, W, stream=S),
    "dense": lambda: m.mla_attend_dense(QT, CACHE, LENS, stream=S),
    "noalloc": lambda: m.mla_attend_dense_noalloc(QT, CACHE, LENS, stream=S),
    "paged": lambda: m.mla_attend_paged(QT, POOL, TABLE, LENS, stream=S),
    "indexed": lambda: m.mla_attend_indexed(QT, CACHE, INDICES, LENS, stream=S),
    "window_dense": lambda: m.mla_attend_window_dense(QT, CACHE, 5, stream=S),
    "window_paged": lambda: m.mla_attend_window_paged(QT, POOL, TABLE, LENS, 5, stream=S),
    "packed": lambda: m.mla_attend_packed(QT, PACKED, TABLE, LENS, stream=S),
    "up_dense": lambda: m.mla_attend_up_dense(QT, CACHE, W, LENS, stream=S),
    "up_paged": lambda: m.mla_attend_up_paged(QT, POOL, TABLE, LENS, W, stream=S),
    "up_indexed": lambda: m.mla_attend_up_indexed(QT, CACHE, INDICES, W, LENS, stream=S),
    "expand_kv": lambda: m.mla_expand_kv(bf(7, 512), W, W, stream=S),
    "prefill": lambda: m.mla_prefill_expanded(bf(1, 4, 64, 256), bf(1, 4, 64, 256), bf(1, 4, 64, 256), stream=S),
    "gather": lambda: m.mla_debug_gather(m.MODE_DENSE, CACHE, i32(4, 3), B=B, stream=S),
    "unpack": lambda: m.mla_cache_unpack(PACKED, TABLE, LENS, 4, stream=S),
    "reserve": lambda: m.mla_pages_reserve(PACKED, TABLE, LENS, REFS, 1, stream=S),
    "fork": lambda: m.mla_pages_fork(PACKED, TABLE, LENS, REFS, i32(1), i32(1), stream=S),
    "compact": lambda: m.mla_pages_compact(PACKED, TABLE, REFS, stream=S),
    "kpool_keys": lambda: m.mla_kpool_keys(CACHE, 64, stream=S),
    "kpool_select": lambda: m.mla_kpool_select(torch.full((B, 2, 512), 0.0), bf(B, Q, 512), 64, 64, stream=S),
    "decode_dense": lambda: m.mla_decode(QH, W, W, CACHE, LENS, stream=S),
    "decode_paged": lambda: m.mla_decode(QH, W, W, POOL, LENS, mode=m.MODE_PAGED, page_table=TABLE, stream=S),
    "decode_indexed": lambda: m.mla_decode(QH, W, W, CACHE, LENS, mode=m.MODE_INDEXED, indices=INDICES, stream=S),
    "decode_fused": lambda: m.mla_decode(QH, W, W, CACHE, LENS, fused=True, stream=S),
    "decode_window": lambda: m.mla_decode(QH, W, W, CACHE, LENS, window=5, stream=S),
    "decode_window_paged": lambda: m.mla_decode(QH, W, W, POOL, LENS, mode=m.MODE_PAGED, page_table=TABLE, window=5, stream=S),
    "decode_packed": lambda: m.mla_decode(QH, W, W, PACKED, LENS, mode=m.MODE_PACKED, page_table=TABLE, stream=S),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_the_streams(monkeypatch, name):
    r = Record(monkeypatch)
    out = CALLS[name]()
    assert r.made and not r.outside, [tuple(t.shape) for t in r.outside]
    for t in out if isinstance(out, tuple) else (out,):
        assert t is None or id(t) in r.read


def _streams(monkeypatch):
    """torch.cuda's current stream, without a device: "caller" until a context changes it."""
    now = ["caller"]

    @contextlib.contextmanager
    def use(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "stream", use)


def test_on_a_stream(monkeypatch):
    """The call runs with the stream as the current one, and its results are recorded for the caller's."""
    _streams(monkeypatch)
    stream, recorded = types.SimpleNamespace(device_index=0), []
    results = tuple(types.SimpleNamespace(record_stream=lambda s, k=k: recorded.append((k, s))) for k in range(2))
    for out, n in ((results, 2), (results[0], 1), ((results[0], None), 1), (None, 0)):
        recorded.clear()
        assert m._on(stream, lambda a, b: (torch.cuda.current_stream(), a, b) == (stream, 1, 2) and out, 1, 2) == out
        assert recorded == [(k, "caller") for k in range(n)]


def test_a_stream_of_another_device_is_refused(monkeypatch):
    _streams(monkeypatch)
    called = []
    with pytest.raises(ValueError, match="the stream is on cuda:1, the current device is cuda:0"):
        m._on(types.SimpleNamespace(device_index=1), called.append, 1)
    assert not called


@pytest.mark.parametrize("name", ["decode_window", "decode_window_paged", "decode_packed"])
def test_decode_launches_nothing_for_another_device(monkeypatch, name):
    """The attention refuses tensors that are not on the current device; q~ is not computed before."""
    launched = []

    class Lib:
        def __getattr__(self, f):
            return lambda *args: launched.append(f) or 0

    check_current = m._check_current
    Record(monkeypatch)
    monkeypatch.setattr(m, "_lib", Lib())
    monkeypatch.setattr(m, "_check_current", check_current)
    monkeypatch.setattr(m, "_check_cuda", lambda *t: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="tensors are on cuda:1, the current device is cuda:0"):
        CALLS[name]()
    assert not launched
