"""Sliding-window attention with sinks over bf16 latent caches, against a plain float64 computation."""
import numpy as np
import pytest
import torch

import mla_absorbed_latent_mtp_b200 as m
import oracle
import synth
from gpu_util import bf16_to_f64, ints_to_dev, synthetic_qtilde, to_dev

pytestmark = pytest.mark.gpu

R, PAGE = 512, 64
NAN = 0x7FC0


@pytest.fixture(scope="module", autouse=True)
def device():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _check(lens, rows, qt_bits, window, sinks, o, lse, scale=1.0 / 16.0):
    """|o - ref| <= 2^-8 |ref| (the bf16 result) + (2^-8 + 2^-13) sum a|c|: the weights are rounded to
    bf16 for the value product; a score is a sum of 512 products in fp32, at most 32 accumulations of
    partial sums below 2^7 that lose 2^-23 each, times the scale 2^-4: 2^-15, so with the
    exponential's 2^-21 a weight and the row sum each move by less than 2^-14."""
    qt = oracle.widen(qt_bits)
    o, lse = bf16_to_f64(o), lse.cpu().numpy().astype(np.float64)
    for b, L in enumerate(lens):
        for i in range(qt.shape[1]):
            at = oracle.window_positions(int(L), qt.shape[1], i, window, sinks)
            ref, ref_lse, mag = oracle.attend_rows(qt[b, i], rows[b][at], scale)
            assert np.isfinite(o[b, i]).all(), (b, i, L)
            err = np.abs(o[b, i] - ref) - (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -13) * mag)
            assert err.max() <= 1e-30, (b, i, L, window, sinks, err.max())
            if at.size == 0:
                assert np.isneginf(lse[b, i]).all()
            else:
                assert np.abs(lse[b, i] - ref_lse).max() <= 2.0 ** -14 + 2.0 ** -22 * np.abs(ref_lse).max()


def _unseen(L, q_len, window, sinks):
    seen = np.zeros(int(L), dtype=bool)
    for i in range(q_len):
        seen[oracle.window_positions(int(L), q_len, i, window, sinks)] = True
    return np.flatnonzero(~seen)


LENS = [1, 300, 64, 65, 127, 128, 129, 63, 257, 1000, 2]
WINDOWS = [(1, 0), (1, 1), (63, 0), (64, 0), (65, 64), (100, 5), (128, 64), (129, 130), (500, 0), (4000, 3), (1, 700), (7, 65)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("q_len", [1, 6])
@pytest.mark.parametrize("paged", [False, True])
def test_windows_match_float64(paged, q_len, window, sinks):
    """Rows that no query sees hold NaN; paged, whole unseen pages are unmapped or out of range."""
    lens = np.array([max(L, q_len) for L in LENS], dtype=np.int32)
    bits = synth.normal_bf16((len(lens), int(lens.max()), R), 1, synth.STREAM_CACHE)
    rows = oracle.widen(bits)
    for b, L in enumerate(lens):
        bits[b, _unseen(L, q_len, window, sinks)] = NAN
        bits[b, L:] = NAN
    qt = synthetic_qtilde(len(lens), q_len, seed=2)
    st = _status()
    if paged:
        table, P = synth.page_layout(lens, 3)
        pool = np.full((P, PAGE, R), NAN, dtype=np.uint16)
        for b, L in enumerate(lens):
            for pg in range(-(-int(L) // PAGE)):
                part = bits[b, pg * PAGE:min((pg + 1) * PAGE, int(L))]
                pool[table[b, pg], :len(part)] = part
                if np.isin(np.arange(pg * PAGE, pg * PAGE + len(part)), _unseen(L, q_len, window, sinks)).all():
                    table[b, pg] = -1 if pg % 2 else 1 << 30
        o, lse = m.mla_attend_window_paged(to_dev(qt), to_dev(pool), ints_to_dev(table), ints_to_dev(lens), window, sinks,
                                           status=st)
    else:
        o, lse = m.mla_attend_window_dense(to_dev(qt), to_dev(bits), window, sinks, ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _check(lens, rows, qt, window, sinks, o, lse)


def test_empty_rows_full_cache_and_scale():
    """Sequences shorter than the query window; seq_lens None (every row of the cache)."""
    lens = np.array([0, 1, 3, 200, 0, 5], dtype=np.int32)
    bits = synth.normal_bf16((len(lens), 200, R), 4, synth.STREAM_CACHE)
    qt = synthetic_qtilde(len(lens), 6, seed=5)
    st = _status()
    o, lse = m.mla_attend_window_dense(to_dev(qt), to_dev(bits), 2, 1, ints_to_dev(lens), scale=0.03, status=st)
    _check(lens, oracle.widen(bits), qt, 2, 1, o, lse, scale=0.03)
    o, lse = m.mla_attend_window_dense(to_dev(qt), to_dev(bits), 70, 4, status=st)
    _check([200] * 6, oracle.widen(bits), qt, 70, 4, o, lse)
    assert int(st.item()) == 0


def test_many_queries_and_many_sequences():
    for lens, q_len, window, sinks in (([300], 300, 50, 3), ([700], 200, 130, 65), ([90 + 5 * b for b in range(200)], 1, 300, 7)):
        lens = np.array(lens, dtype=np.int32)
        bits = synth.normal_bf16((len(lens), int(lens.max()), R), 6, synth.STREAM_CACHE)
        qt = synthetic_qtilde(len(lens), q_len, seed=7)
        st = _status()
        o, lse = m.mla_attend_window_dense(to_dev(qt), to_dev(bits), window, sinks, ints_to_dev(lens), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        _check(lens, oracle.widen(bits), qt, window, sinks, o, lse)


def test_a_window_over_everything_is_dense_attention():
    """Same tiles, same split: the weights differ only in whether the sum takes them rounded."""
    lens = np.array([1000, 333, 64], dtype=np.int32)
    bits = synth.normal_bf16((3, 1000, R), 8, synth.STREAM_CACHE)
    qt = to_dev(synthetic_qtilde(3, 2, seed=9))
    o0, lse0 = m.mla_attend_dense(qt, to_dev(bits), ints_to_dev(lens))
    for window, sinks in ((1000, 0), (2**31 - 1, 2**31 - 1)):
        o1, lse1 = m.mla_attend_window_dense(qt, to_dev(bits), window, sinks, ints_to_dev(lens))
        # both sums are within 2^-8 of each other; two bf16 results of values that close
        assert ((o1.float() - o0.float()).abs() <= 2.0 ** -8 * 3 * o0.float().abs() + 1e-6).all()
        assert (lse1 - lse0).abs().max() <= 2.0 ** -8


def test_rising_scores_rescale_inside_the_window():
    lens = np.array([900], dtype=np.int32)
    qt_bits = synthetic_qtilde(1, 1, seed=10)
    qt = oracle.widen(qt_bits)
    rows = oracle.widen(synth.normal_bf16((1, 900, R), 11, synth.STREAM_CACHE))
    rows += (np.arange(900) / 150.0)[None, :, None] * np.sign(qt[0, 0, 3])[None, None]
    bits = synth.f64_to_bf16_bits(rows)
    rows = oracle.widen(bits)
    st = _status()
    o, lse = m.mla_attend_window_dense(to_dev(qt_bits), to_dev(bits), 700, 10, ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    at = oracle.window_positions(900, 1, 0, 700, 10)
    ref, ref_lse, mag = oracle.attend_rows(qt[0, 0], rows[0][at])
    # as _check, with partial sums up to the largest sum of |q c|
    s = (np.abs(qt[0, 0]) @ np.abs(rows[0][at]).T / 16).max(axis=1, keepdims=True)
    rel = 2.0 ** -8 + 2 * s * 32 * 2.0 ** -23 + 2.0 ** -20
    assert (np.abs(bf16_to_f64(o)[0, 0] - ref) <= 2.0 ** -8 * np.abs(ref) + rel * mag + 1e-30).all()
    assert (np.abs(lse.cpu().numpy()[0, 0] - ref_lse) <= 2 * s[:, 0] * 32 * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref_lse)).all()


def test_bad_pages_and_lengths_are_flagged():
    lens = np.array([200, 200], dtype=np.int32)
    table, P = synth.page_layout(lens, 12)
    pool = to_dev(synth.normal_bf16((P, PAGE, R), 12, synth.STREAM_CACHE))
    qt = to_dev(synthetic_qtilde(2, 1, seed=13))
    st = _status()
    for bad in (-1, P, 1 << 30):
        t2 = table.copy()
        t2[1, 3] = bad
        st.zero_()
        m.mla_attend_window_paged(qt, pool, ints_to_dev(t2), ints_to_dev(lens), 100, 3, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == m.MLA_ERR_INDEX
    st.zero_()
    m.mla_attend_window_paged(qt, pool, ints_to_dev(table), ints_to_dev([200, 4 * PAGE + 1]), 100, 3, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == m.MLA_ERR_INDEX


@pytest.mark.parametrize("q_len,lens,window,sinks", [(1, [1], 1, 0), (1, [12000], 20000, 0), (1, [12000], 3000, 70), (6, [2500], 900, 3),
                                                     (1, [700] * 9, 800, 0), (8, [118] * 25, 50, 4), (1, [100] * 148, 70, 0),
                                                     (1, [k % 5 * 70 for k in range(160)], 100, 1)])
def test_merges_read_only_what_the_call_wrote(q_len, lens, window, sinks):
    """The workspace holds NaN before the call; twice, with the first call's contents before the second."""
    lens = np.array(lens, dtype=np.int32)
    bits = synth.normal_bf16((len(lens), max(int(lens.max()), 1), R), 33, synth.STREAM_CACHE)
    qt = synthetic_qtilde(len(lens), q_len, seed=34)
    ws = m.new_workspace(len(lens), q_len)
    ws.fill_(0xFF)
    st = _status()
    args = (to_dev(qt), to_dev(bits), window, sinks, ints_to_dev(lens))
    o, lse = m.mla_attend_window_dense(*args, workspace=ws, status=st)
    again, lse_again = m.mla_attend_window_dense(*args, workspace=ws, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(o, again) and torch.equal(lse, lse_again)
    _check(lens, oracle.widen(bits), qt, window, sinks, o, lse)


# Every form of the merge, a tile per CTA: a single row; few sequences; more; as many as CTA groups.
TILE_EACH = [[6401], [3201, 3200], [129] * 20, [129] * 40 + [0] * 110]


def _aligned(lens, seed):
    """Head 0 of every sequence scores 200 and more at row 3 and about 0 elsewhere: every partial but the
    first tile's has the weight 2^-288 or less, zero in fp32."""
    bits = synth.normal_bf16((len(lens), max(lens), R), seed, synth.STREAM_CACHE, 0.01)
    qt = synthetic_qtilde(len(lens), 1, seed=seed + 1)
    q = oracle.widen(qt)[:, 0, 0]
    assert (q != 0).all() and np.abs(q).sum(axis=1).min() > 200
    bits[:, 3] = synth.f64_to_bf16_bits(np.sign(q) * 16.0)
    return bits, qt, q


def _finite_but_first(lens, o, lse):
    assert torch.isfinite(o[1:].float()).all() and not torch.isnan(lse[1:]).any()
    assert torch.isfinite(lse[1:][ints_to_dev(lens)[1:] > 0]).all()


@pytest.mark.parametrize("lens", TILE_EACH)
def test_a_nan_query_gives_nan(lens):
    """The whole head, and no other."""
    bits = synth.normal_bf16((len(lens), max(lens), R), 40, synth.STREAM_CACHE)
    qt = synthetic_qtilde(len(lens), 1, seed=41)
    bad = qt.copy()
    bad[0, 0, 5, 100] = NAN
    args = (to_dev(bits), 1000, 3, ints_to_dev(lens))
    st = _status()
    want, lse_want = m.mla_attend_window_dense(to_dev(qt), *args, status=st)
    o, lse = m.mla_attend_window_dense(to_dev(bad), *args, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.isnan(o[0, 0, 5]).all() and torch.isnan(lse[0, 0, 5])
    o[0, 0, 5], lse[0, 0, 5] = want[0, 0, 5], lse_want[0, 0, 5]
    _check(lens[:2], oracle.widen(bits[:2]), qt[:2], 1000, 3, o[:2], lse[:2])


@pytest.mark.parametrize("window", [1, 64, 100000])
@pytest.mark.parametrize("lens", TILE_EACH)
def test_a_nan_in_a_seen_row_gives_nan(lens, window):
    """The only seen row of its tile and CTA."""
    bits = synth.normal_bf16((len(lens), max(lens), R), 42, synth.STREAM_CACHE)
    bits[0, lens[0] - 1, 77] = NAN
    qt = synthetic_qtilde(len(lens), 1, seed=43)
    st = _status()
    o, lse = m.mla_attend_window_dense(to_dev(qt), to_dev(bits), window, 0, ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    _finite_but_first(lens, o, lse)


@pytest.mark.parametrize("alone", [False, True])
@pytest.mark.parametrize("lens", TILE_EACH)
def test_a_nan_survives_a_weight_of_zero(lens, alone):
    """In a row (alone: the only one of its tile) that counts for nothing beside another tile's: 0 x NaN."""
    bits, qt, _ = _aligned(lens, 44)
    bits[0, lens[0] - 1 if alone else 100, 200] = NAN
    st = _status()
    o, lse = m.mla_attend_window_dense(to_dev(qt), to_dev(bits), 100000, 0, ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    _finite_but_first(lens, o, lse)


@pytest.mark.parametrize("alone", [False, True])
@pytest.mark.parametrize("lens", TILE_EACH)
def test_an_infinite_row_of_weight_zero_gives_nan(lens, alone):
    """Its score is -Inf for head 0: weight 0, and 0 x Inf in every latent; lse is that of the other rows."""
    bits, qt, q = _aligned(lens, 46)
    bits[0, lens[0] - 1 if alone else 100] = np.where(q[0] > 0, 0xFF80, 0x7F80)
    st = _status()
    o, lse = m.mla_attend_window_dense(to_dev(qt), to_dev(bits), 100000, 0, ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.isnan(o[0, 0, 0]).all() and torch.isfinite(lse[0, 0, 0])
    _finite_but_first(lens, o, lse)


@pytest.mark.parametrize("window,sinks", [(1000, 0), (2**31 - 1, 2**31 - 1)])
def test_a_window_over_everything_matches_float64(window, sinks):
    lens = np.array([1000, 333, 64], dtype=np.int32)
    bits = synth.normal_bf16((3, 1000, R), 8, synth.STREAM_CACHE)
    qt = synthetic_qtilde(3, 2, seed=9)
    st = _status()
    o, lse = m.mla_attend_window_dense(to_dev(qt), to_dev(bits), window, sinks, ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _check(lens, oracle.widen(bits), qt, 0, 0, o, lse)


def _step_inputs(seed, n):
    lens = np.array([900 + 50 * n, 64, 5, 333], dtype=np.int32)
    table, P = synth.page_layout(lens, seed)
    pool = to_dev(synth.normal_bf16((P, PAGE, R), seed, synth.STREAM_CACHE))
    return to_dev(synthetic_qtilde(4, 2, seed=seed + 1)), pool, ints_to_dev(table), ints_to_dev(lens)


def test_captured_and_replayed():
    """Dense and paged calls in one graph, with short and empty lists, replayed on other lengths and queries."""
    qt, pool, table, lens = _step_inputs(50, 0)
    cache = to_dev(synth.normal_bf16((4, 950, R), 52, synth.STREAM_CACHE))
    ws, st = m.new_workspace(4, 2), _status()

    def step():
        return (*m.mla_attend_window_paged(qt, pool, table, lens, 100, 3, workspace=ws, status=st),
                *m.mla_attend_window_dense(qt, cache, 300, 0, lens, workspace=ws, status=st))

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for k, now in enumerate(([900, 64, 5, 333], [900, 0, 0, 1], [0, 0, 0, 0], [2, 64, 5, 200])):
        lens.copy_(ints_to_dev(now))
        qt.copy_(to_dev(synthetic_qtilde(4, 2, seed=53 + k)))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        for x, y in zip(got, step()):
            assert torch.equal(x, y)
    assert int(st.item()) == 0


def test_two_streams_at_once():
    """Each with its own workspace, and lists so short that most CTAs have nothing to load."""
    inputs = [_step_inputs(60, 0), _step_inputs(62, 1)]
    wss = [m.new_workspace(4, 2) for _ in inputs]
    sts = [_status() for _ in inputs]
    alone = [m.mla_attend_window_paged(*x, 100, 3, workspace=ws) for x, ws in zip(inputs, wss)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(20):
        got = []
        for x, ws, st, s in zip(inputs, wss, sts, streams):
            with torch.cuda.stream(s):
                got.append(m.mla_attend_window_paged(*x, 100, 3, workspace=ws, status=st))
        torch.cuda.synchronize()
        for x, y, st in zip(got, alone, sts):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]) and int(st.item()) == 0
