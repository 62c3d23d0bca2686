"""The windowed, packed and page entry points refuse bad host-side arguments before touching the
device (C ABI), and tensors whose dtype, layout or size would let a kernel address memory outside
them (binding).  None of these calls launches anything."""
import ctypes

import numpy as np
import pytest
import torch

import mla_absorbed_latent_mtp_b200 as m

P = ctypes.c_void_p
GOOD, ODD = P(1 << 20), P((1 << 20) + 8)
ARG, UNSUPPORTED, WORKSPACE = m.MLA_ERR_ARG, m.MLA_ERR_UNSUPPORTED, m.MLA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return m.lib()


def caller(f, order, good):
    def call(**kw):
        a = dict(good, **kw)
        assert set(a) == set(order.split())
        return f(*(a[k] for k in order.split()))
    return call


def test_status_of_a_full_pool(lib):
    assert m.status_string(m.MLA_ERR_PAGES) == "MLA_ERR_PAGES"


def test_window_dense(lib):
    call = caller(lib.mla_attend_window_dense, "qt c lens B Q H R L s w k ws wsb o lse st stream",
                  dict(qt=GOOD, c=GOOD, lens=None, B=1, Q=1, H=64, R=512, L=8, s=0.0625, w=4, k=0, ws=GOOD, wsb=1 << 30,
                       o=GOOD, lse=None, st=None, stream=None))
    for kw in (dict(qt=None), dict(c=None), dict(o=None), dict(B=0), dict(Q=0), dict(L=0), dict(w=0), dict(w=-1), dict(k=-1),
               dict(s=float("inf")), dict(L=2**31 - 64), dict(B=1 << 15, L=1 << 16)):
        assert call(**kw) == ARG, kw
    for kw in (dict(H=32), dict(R=576), dict(c=ODD), dict(qt=ODD), dict(o=ODD)):
        assert call(**kw) == UNSUPPORTED, kw


def test_window_paged(lib):
    call = caller(lib.mla_attend_window_paged, "qt c t lens B Q H R page mp np s w k ws wsb o lse st stream",
                  dict(qt=GOOD, c=GOOD, t=GOOD, lens=GOOD, B=1, Q=1, H=64, R=512, page=64, mp=4, np=4, s=0.0625, w=4, k=0,
                       ws=GOOD, wsb=1 << 30, o=GOOD, lse=None, st=None, stream=None))
    for kw in (dict(t=None), dict(lens=None), dict(mp=0), dict(np=0), dict(w=0), dict(k=-1), dict(mp=1 << 25),
               dict(mp=(1 << 25) - 1), dict(np=1 << 25)):
        assert call(**kw) == ARG, kw
    assert call(page=32) == UNSUPPORTED


def test_packed_attend(lib):
    call = caller(lib.mla_attend_packed, "qt c t lens B Q H R page mp np u w k s ws wsb o lse st stream",
                  dict(qt=GOOD, c=GOOD, t=GOOD, lens=GOOD, B=1, Q=1, H=64, R=512, page=64, mp=4, np=4, u=1.0, w=0, k=0,
                       s=0.0625, ws=GOOD, wsb=1 << 30, o=GOOD, lse=None, st=None, stream=None))
    for kw in (dict(qt=None), dict(c=None), dict(t=None), dict(lens=None), dict(o=None), dict(B=0), dict(Q=0), dict(mp=0),
               dict(np=0), dict(w=-1), dict(k=-1), dict(s=float("nan")), dict(mp=(1 << 25) - 2), dict(np=1 << 25),
               dict(B=1 << 20, Q=1 << 5)):
        assert call(**kw) == ARG, kw
    for unit in (0.0, -1.0, 3.0, float("inf"), float("nan"), 2.0 ** 65, 2.0 ** -65, 1e-45):
        assert call(u=unit) == ARG, unit
    for kw in (dict(H=32), dict(R=576), dict(page=32), dict(c=ODD), dict(qt=ODD), dict(o=ODD)):
        assert call(**kw) == UNSUPPORTED, kw


def test_packed_cache(lib):
    call = caller(lib.mla_cache_append_packed, "pool t lens rows B Q R page mp np u st stream",
                  dict(pool=GOOD, t=GOOD, lens=GOOD, rows=GOOD, B=1, Q=1, R=512, page=64, mp=4, np=4, u=1.0, st=None,
                       stream=None))
    for kw in (dict(pool=None), dict(t=None), dict(lens=None), dict(rows=None), dict(B=0), dict(Q=0), dict(mp=0), dict(np=0),
               dict(u=1.5), dict(mp=1 << 25), dict(np=1 << 25), dict(Q=32 * 65535 + 1)):
        assert call(**kw) == ARG, kw
    for kw in (dict(R=256), dict(page=128), dict(pool=ODD), dict(rows=ODD)):
        assert call(**kw) == UNSUPPORTED, kw
    call = caller(lib.mla_cache_truncate_packed, "pool t lens keep B Q R page mp np st stream",
                  dict(pool=GOOD, t=GOOD, lens=GOOD, keep=GOOD, B=1, Q=1, R=512, page=64, mp=4, np=4, st=None, stream=None))
    for kw in (dict(pool=None), dict(keep=None), dict(lens=None), dict(B=0), dict(Q=0)):
        assert call(**kw) == ARG, kw
    assert call(R=64) == UNSUPPORTED
    call = caller(lib.mla_cache_unpack, "pool t start rows B n R page mp np u st stream",
                  dict(pool=GOOD, t=GOOD, start=GOOD, rows=GOOD, B=1, n=1, R=512, page=64, mp=4, np=4, u=1.0, st=None,
                       stream=None))
    for kw in (dict(pool=None), dict(start=None), dict(rows=None), dict(n=0), dict(u=0.3)):
        assert call(**kw) == ARG, kw
    for kw in (dict(rows=ODD), dict(B=65536)):
        assert call(**kw) == UNSUPPORTED, kw


def test_pages(lib):
    ws = lib.mla_pages_workspace_bytes
    assert ws(0, 4) == 0 and ws(4, 0) == 0 and ws(4, 1 << 25) == 0
    assert 0 < ws(1, 1) < ws(1000, 1) < ws(1000, 1 << 20)
    good = dict(pool=GOOD, pb=64, t=GOOD, lens=GOOD, refs=GOOD, B=2, mp=4, np=8, ws=GOOD, wsb=1 << 20, st=None, stream=None)
    reserve = caller(lib.mla_pages_reserve, "pool pb t lens refs B Q mp np ws wsb st stream", dict(good, Q=1))
    fork = caller(lib.mla_pages_fork, "pool pb t lens refs par kid n B mp np ws wsb st stream",
                  dict(good, par=GOOD, kid=GOOD, n=1))
    none = {k: v for k, v in good.items() if k != "lens"}
    compact = caller(lib.mla_pages_compact, "pool pb t refs B mp np used ws wsb st stream", dict(none, used=GOOD))
    for call in (reserve, fork, compact):
        for kw in (dict(pool=None), dict(t=None), dict(refs=None), dict(B=0), dict(mp=0), dict(np=0), dict(mp=1 << 25),
                   dict(np=1 << 25)):
            assert call(**kw) == ARG, kw
        for kw in (dict(pb=8), dict(pb=40), dict(pool=ODD)):
            assert call(**kw) == UNSUPPORTED, kw
        for kw in (dict(ws=None), dict(wsb=16), dict(ws=ODD)):
            assert call(**kw) == WORKSPACE, kw
    assert reserve(lens=None) == ARG and reserve(Q=0) == ARG
    assert fork(par=None) == ARG and fork(kid=None) == ARG and fork(n=0) == ARG and fork(lens=None) == ARG
    assert compact(used=None) == ARG
    release = caller(lib.mla_pages_release, "t lens refs B mp np st stream",
                     dict(t=GOOD, lens=GOOD, refs=GOOD, B=2, mp=4, np=8, st=None, stream=None))
    for kw in (dict(t=None), dict(lens=None), dict(refs=None), dict(B=0), dict(mp=0), dict(np=0)):
        assert release(**kw) == ARG, kw


# ----------------------------------------------------------------------------- the binding
def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def _refused(fn, *args, match, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_window_binding(lib):
    qt, cache, pool, table, lens = bf(2, 1, 64, 512), bf(2, 130, 512), bf(5, 64, 512), i32(2, 3), i32(2)
    _refused(m.mla_attend_window_dense, qt, bf(1, 130, 512), 8, match="cache holds 1 sequences")
    _refused(m.mla_attend_window_dense, qt, cache.float(), 8, match="cache must be")
    _refused(m.mla_attend_window_dense, qt, cache, 8, 0, i32(1), match="seq_lens needs at least 2")
    _refused(m.mla_attend_window_dense, qt, cache, 8, match="CUDA tensors")
    _refused(m.mla_attend_window_paged, qt, bf(5, 32, 512), table, lens, 8, match="pool must have shape")
    _refused(m.mla_attend_window_paged, qt, pool, i32(1, 3), lens, 8, match="page_table has 1 rows")
    _refused(m.mla_attend_window_paged, qt, pool, table, None, 8, match="seq_lens is required")
    _refused(m.mla_attend_window_paged, qt, pool, table, lens, 8, workspace=u8(16), match="workspace needs at least")
    _refused(m.mla_attend_window_paged, qt, pool, table, lens, 8, match="CUDA tensors")


def test_packed_binding(lib):
    qt, pool, table, lens, rows = bf(2, 1, 64, 512), u8(5, 64, 288), i32(2, 3), i32(2), bf(2, 6, 512)
    _refused(m.mla_attend_packed, qt, u8(5, 64, 256), table, lens, match="pool must have shape")
    _refused(m.mla_attend_packed, qt, bf(5, 64, 288), table, lens, match="pool must be")
    _refused(m.mla_attend_packed, qt, u8(5, 64, 576)[:, :, ::2], table, lens, match="pool must be contiguous")
    _refused(m.mla_attend_packed, qt, pool, i32(1, 3), lens, match="page_table has 1 rows")
    _refused(m.mla_attend_packed, qt, pool, table, None, match="seq_lens is required")
    _refused(m.mla_attend_packed, qt, pool, table, lens, match="CUDA tensors")
    _refused(m.mla_cache_append_packed, pool, table, i32(1), rows, match="seq_lens needs at least")
    _refused(m.mla_cache_append_packed, pool, table, lens, bf(2, 6, 256), match="rows must have shape")
    _refused(m.mla_cache_append_packed, pool, table, lens, rows, match="CUDA tensors")
    _refused(m.mla_cache_truncate_packed, pool, table, lens, i32(1), 6, match="keep needs at least")
    _refused(m.mla_cache_truncate_packed, pool, i32(1, 3), lens, i32(2), 6, match="page_table has 1 rows")
    _refused(m.mla_cache_unpack, pool, table, lens, 6, rows=bf(2, 5, 512), match="rows must have shape")
    _refused(m.mla_cache_unpack, pool, table, lens, 6, match="CUDA tensors")
    q, w = bf(2, 1, 64, 256), bf(64, 256, 512)
    _refused(m.mla_decode, q, w, w, pool, lens, mode=m.MODE_PACKED, page_table=table, fused=True, match="no windowed or packed")
    _refused(m.mla_decode, q, w, w, pool, lens, mode=m.MODE_INDEXED, window=3, match="no window")


def test_pages_binding(lib):
    pool, table, lens, refs = u8(5, 64, 288), i32(2, 3), i32(2), i32(5)
    _refused(m.mla_pages_reserve, pool, table.long(), lens, refs, 1, match="page_table must be")
    _refused(m.mla_pages_reserve, pool, table, i32(1), refs, 1, match="seq_lens needs at least")
    _refused(m.mla_pages_reserve, pool, table, lens, i32(4), 1, match="one element per page")
    _refused(m.mla_pages_reserve, u8(5, 32, 288), table, lens, refs, 1, match="pool must be a contiguous")
    _refused(m.mla_pages_reserve, u8(5, 64, 576)[:, :, ::2], table, lens, refs, 1, match="pool must be a contiguous")
    _refused(m.mla_pages_reserve, pool, table, lens, refs, 1, workspace=u8(4), match="workspace needs at least")
    _refused(m.mla_pages_reserve, pool, table, lens, refs, 1, match="CUDA tensors")
    _refused(m.mla_pages_fork, pool, table, lens, refs, i32(2), i32(1), match="children must have shape")
    _refused(m.mla_pages_fork, pool, table, lens, refs, i32(1), i32(1), match="CUDA tensors")
    _refused(m.mla_pages_release, table, lens, refs.long(), match="refs must be")
    _refused(m.mla_pages_release, table, lens, refs, match="CUDA tensors")
    _refused(m.mla_pages_compact, pool, table, refs, n_used=torch.zeros(1), match="n_used must be")
    _refused(m.mla_pages_compact, pool, table, refs, match="CUDA tensors")


@pytest.mark.parametrize("big", [2**31, 2**32 + 1, -2**31 - 1])
def test_numbers_past_32_bits(lib, big):
    """Refused by name, before anything else is looked at: they would wrap to another number."""
    for name, call in (("window", lambda: m.mla_attend_window_dense(None, None, big)),
                       ("sinks", lambda: m.mla_attend_window_dense(None, None, 4, big)),
                       ("window", lambda: m.mla_attend_window_paged(None, None, None, None, big)),
                       ("sinks", lambda: m.mla_attend_window_paged(None, None, None, None, 4, big)),
                       ("window", lambda: m.mla_attend_packed(None, None, None, None, window=big)),
                       ("sinks", lambda: m.mla_attend_packed(None, None, None, None, sinks=big)),
                       ("q_len", lambda: m.mla_cache_truncate_packed(None, None, None, None, big)),
                       ("n", lambda: m.mla_cache_unpack(None, None, None, big)),
                       ("q_len", lambda: m.mla_pages_reserve(None, None, None, None, big)),
                       ("num_pages", lambda: m.mla_pages_workspace_bytes(1, big)),
                       ("n", lambda: m.mla_pages_workspace_bytes(big, 1))):
        with pytest.raises(ValueError, match=f"^{name} must fit 32 bits"):
            call()


@pytest.mark.parametrize("big", [2**31, 2**32 + 1, -2**31 - 1])
def test_numpy_and_tensor_numbers_past_32_bits(lib, big):
    """They have no Python int's type, and ctypes wraps them all the same."""
    for make in (np.int64, torch.tensor):
        for name, call in (("window", lambda: m.mla_attend_window_dense(None, None, make(big))),
                           ("sinks", lambda: m.mla_attend_packed(None, None, None, None, sinks=make(big))),
                           ("q_len", lambda: m.mla_pages_reserve(None, None, None, None, make(big))),
                           ("n", lambda: m.mla_pages_workspace_bytes(make(big), 1))):
            with pytest.raises(ValueError, match=f"^{name} must fit 32 bits"):
                call()
    assert m.mla_pages_workspace_bytes(np.int64(3), np.int32(5)) == m.mla_pages_workspace_bytes(3, 5)
