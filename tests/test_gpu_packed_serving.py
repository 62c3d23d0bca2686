"""The 4-bit cache as a serving loop uses it: reserve, quantising append, verify, roll back, release,
fork, attend inside a window, compact -- each state against the oracle -- and the same steps
captured into CUDA graphs, on other streams, and two at a time."""
import numpy as np
import pytest
import torch

import mla_absorbed_latent_mtp_b200 as m
import oracle
import synth
from gpu_util import ints_to_dev, synthetic_qtilde, to_dev
from test_gpu_packed import _check, _rows

pytestmark = pytest.mark.gpu

PAGE, ROW = 64, 288


@pytest.fixture(scope="module", autouse=True)
def device():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


class Cache:
    def __init__(self, B, max_pages, P):
        dev = dict(dtype=torch.int32, device="cuda")
        self.pool = torch.zeros(P, PAGE, ROW, dtype=torch.uint8, device="cuda")
        self.table = torch.full((B, max_pages), -1, **dev)
        self.lens, self.refs = torch.zeros(B, **dev), torch.zeros(P, **dev)
        self.status = torch.zeros(1, **dev)
        self.ws = m.new_pages_workspace(B, P)
        self.rows = [np.zeros((0, 512)) for _ in range(B)]  # the float64 values that the cache stands for

    def append(self, bits, unit=1.0):
        B, Q = bits.shape[:2]
        m.mla_pages_reserve(self.pool, self.table, self.lens, self.refs, Q, workspace=self.ws, status=self.status)
        m.mla_cache_append_packed(self.pool, self.table, self.lens, to_dev(bits), unit=unit, status=self.status)
        v = oracle.packed_values(oracle.packed_quantise(oracle.widen(bits), unit), unit)
        for b in range(B):
            self.rows[b] = np.concatenate([self.rows[b], v[b]])

    def truncate(self, keep, q_len):
        m.mla_cache_truncate_packed(self.pool, self.table, self.lens, ints_to_dev(keep), q_len, status=self.status)
        m.mla_pages_release(self.table, self.lens, self.refs, status=self.status)
        for b, k in enumerate(keep):
            self.rows[b] = self.rows[b][:len(self.rows[b]) - q_len + k]

    def check(self, qt, window=0, sinks=0):
        o, lse = m.mla_attend_packed(to_dev(qt), self.pool, self.table, self.lens, window=window, sinks=sinks,
                                     status=self.status)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0, m.status_string(int(self.status.item()))
        lens = [len(r) for r in self.rows]
        assert self.lens.cpu().tolist() == lens
        _check(lens, self.rows, qt, window, sinks, o, lse)


def test_serving_loop():
    B, q_len = 5, 6
    c = Cache(B, 8, 48)
    c.append(_rows((B, 100), 1))
    for step in range(4):
        c.append(_rows((B, q_len), 10 + step))
        c.check(synthetic_qtilde(B, q_len, seed=step))
        c.truncate([step % 7, 6, 0, 3, 1], q_len)
        c.check(synthetic_qtilde(B, 1, seed=20 + step), window=50, sinks=4)
    # sequence 4 ends; sequence 0 is forked into its place; both go on
    c.lens[4] = 0
    c.rows[4] = c.rows[0].copy()
    m.mla_pages_release(c.table, c.lens, c.refs, status=c.status)
    m.mla_pages_fork(c.pool, c.table, c.lens, c.refs, ints_to_dev([0]), ints_to_dev([4]), workspace=c.ws, status=c.status)
    c.check(synthetic_qtilde(B, 1, seed=30))
    c.append(_rows((B, q_len), 31))
    c.check(synthetic_qtilde(B, q_len, seed=32))
    c.check(synthetic_qtilde(B, q_len, seed=33), window=20, sinks=1)
    n = m.mla_pages_compact(c.pool, c.table, c.refs, workspace=c.ws, status=c.status)
    c.check(synthetic_qtilde(B, 2, seed=34))
    n = int(n.item())
    assert n == int((c.refs > 0).sum().item()) and int(c.table.max().item()) < n and not c.refs[n:].any()
    # the packed values go back into the expanded form
    start = ints_to_dev([0] * B)
    n_rows = min(len(r) for r in c.rows)
    back = m.mla_cache_unpack(c.pool, c.table, start, n_rows, status=c.status)
    assert np.array_equal(back.float().cpu().numpy().astype(np.float64), np.stack([r[:n_rows] for r in c.rows]))


def test_whole_path_through_mla_decode():
    B = 3
    c = Cache(B, 4, 16)
    c.append(_rows((B, 150), 40))
    w = [to_dev(synth.normal_bf16((64, 256, 512), 41, s, 512 ** -0.5)) for s in (synth.STREAM_WUK, synth.STREAM_WUV)]
    q = to_dev(synth.normal_bf16((B, 1, 64, 256), 42, synth.STREAM_Q))
    got, lse = m.mla_decode(q, *w, c.pool, c.lens, mode=m.MODE_PACKED, page_table=c.table, window=64, sinks=2)
    o, lse2 = m.mla_attend_packed(m.mla_absorb_q(q, w[0]), c.pool, c.table, c.lens, window=64, sinks=2)
    assert torch.equal(got, m.mla_up_proj(o, w[1])) and torch.equal(lse, lse2)
    bf = to_dev(_rows((B, 150), 43))
    got, _ = m.mla_decode(q, *w, bf, mode=m.MODE_DENSE, window=64, sinks=2)
    o, _ = m.mla_attend_window_dense(m.mla_absorb_q(q, w[0]), bf, 64, 2)
    assert torch.equal(got, m.mla_up_proj(o, w[1]))


def test_captured_and_replayed():
    """One captured serving step, replayed: the same bits as the calls made one by one."""
    B, q_len = 4, 3
    def build():
        c = Cache(B, 8, 40)
        c.append(_rows((B, 77), 50))
        return c
    a, g = build(), build()
    rows = to_dev(_rows((B, q_len), 51))
    qt = to_dev(synthetic_qtilde(B, q_len, seed=52))
    ws = m.new_workspace(B, q_len)
    keep = ints_to_dev([1, 3, 0, 2])

    def step(c):
        m.mla_pages_reserve(c.pool, c.table, c.lens, c.refs, q_len, workspace=c.ws, status=c.status)
        m.mla_cache_append_packed(c.pool, c.table, c.lens, rows, status=c.status)
        o, lse = m.mla_attend_packed(qt, c.pool, c.table, c.lens, window=40, sinks=3, workspace=ws, status=c.status)
        m.mla_cache_truncate_packed(c.pool, c.table, c.lens, keep, q_len, status=c.status)
        m.mla_pages_release(c.table, c.lens, c.refs, status=c.status)
        return o, lse

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = step(g)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        want = step(a)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        for x, y in ((a.pool, g.pool), (a.table, g.table), (a.lens, g.lens), (a.refs, g.refs)):
            assert torch.equal(x, y)
    assert int(a.status.item()) == 0 and int(g.status.item()) == 0


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give the bits of one call alone."""
    caches, alone, qts, wss = [], [], [], []
    for k in range(2):
        c = Cache(6, 20, 130)
        c.append(_rows((6, 900 + 100 * k), 60 + k))
        qt = to_dev(synthetic_qtilde(6, 2, seed=62 + k))
        caches.append(c)
        qts.append(qt)
        wss.append(m.new_workspace(6, 2))
        alone.append(m.mla_attend_packed(qt, c.pool, c.table, c.lens, workspace=wss[-1]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = []
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                c = caches[k]
                got.append(m.mla_attend_packed(qts[k], c.pool, c.table, c.lens, workspace=wss[k], status=c.status))
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(got[k][0], alone[k][0]) and torch.equal(got[k][1], alone[k][1])
            assert int(caches[k].status.item()) == 0


def test_stream_argument():
    c = Cache(2, 4, 12)
    c.append(_rows((2, 130), 70))
    qt = to_dev(synthetic_qtilde(2, 1, seed=71))
    want = m.mla_attend_packed(qt, c.pool, c.table, c.lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = m.new_workspace(2, 1)
    got = m.mla_attend_packed(qt, c.pool, c.table, c.lens, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_outputs_of_a_call_on_another_stream_are_not_memory_that_is_still_written():
    """A tensor of the outputs' size is freed while a copy into it waits on the current stream; a
    call on another stream makes its outputs meanwhile."""
    c = Cache(2, 4, 12)
    c.append(_rows((2, 130), 72))
    qt = to_dev(synthetic_qtilde(2, 1, seed=73))
    ws = m.new_workspace(2, 1)
    want = m.mla_attend_packed(qt, c.pool, c.table, c.lens, workspace=ws)
    rows = m.mla_cache_unpack(c.pool, c.table, torch.zeros_like(c.lens), 130)
    torch.cuda.synchronize()
    start = torch.zeros_like(c.lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    gate = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")  # some milliseconds of fills
    late = [torch.empty_like(x) for x in (*want, rows)]
    for _ in range(60):
        gate.zero_()
    for x in late:
        x.zero_()
    del late, x
    got = m.mla_attend_packed(qt, c.pool, c.table, c.lens, workspace=ws, stream=s)
    got_rows = m.mla_cache_unpack(c.pool, c.table, start, 130, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got_rows, rows)


@pytest.mark.parametrize("late", ["current", "side"])
@pytest.mark.parametrize("form", ["packed", "window", "window_paged", "dense", "paged", "fused"])
def test_decode_on_another_stream(form, late):
    """mla_decode's own tensors are the stream's.  The current stream still writes freed tensors of
    their sizes when the call is made (late = current), or the call's stream is behind and the current one
    fills new tensors of their sizes meanwhile (late = side)."""
    B = 2
    c = Cache(B, 4, 12)
    c.append(_rows((B, 130), 74))
    w = [to_dev(synth.normal_bf16((64, 256, 512), 75, s, 512 ** -0.5)) for s in (synth.STREAM_WUK, synth.STREAM_WUV)]
    q = to_dev(synth.normal_bf16((B, 1, 64, 256), 76, synth.STREAM_Q))
    cache, pool = to_dev(_rows((B, 130), 77)), to_dev(_rows((12, PAGE), 78))
    args, kw = {"packed": ((c.pool, c.lens), dict(mode=m.MODE_PACKED, page_table=c.table, window=64)),
                "window": ((cache, c.lens), dict(window=64, sinks=2)),
                "window_paged": ((pool, c.lens), dict(mode=m.MODE_PAGED, page_table=c.table, window=64)),
                "dense": ((cache, c.lens), {}),
                "paged": ((pool, c.lens), dict(mode=m.MODE_PAGED, page_table=c.table)),
                "fused": ((cache, c.lens), dict(fused=True))}[form]
    want = m.mla_decode(q, *w, *args, **kw, status=c.status)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    gate = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")  # some milliseconds of fills
    own = [torch.empty(B, 1, 64, n, dtype=torch.bfloat16, device="cuda") for n in (512, 512, 256)]
    own += [torch.empty_like(want[1]), torch.empty_like(m.new_workspace(B, 1))]
    shapes = [(x.shape, x.dtype) for x in own]
    with torch.cuda.stream(torch.cuda.current_stream() if late == "current" else s):
        for _ in range(60):
            gate.zero_()
    if late == "current":
        for x in own:
            x.fill_(255)
        del x
    own = None
    got = m.mla_decode(q, *w, *args, **kw, status=c.status, stream=s)
    if late == "side":
        own = [torch.full(shape, 255, dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
