"""The 4-bit latent cache on the GPU: append, truncate and read-back bit for bit against the
oracle, attention against a plain float64 computation on the same packed rows."""
import numpy as np
import pytest
import torch

import mla_absorbed_latent_mtp_b200 as m
import oracle
import synth
from gpu_util import bf16_to_f64, ints_to_dev, synthetic_qtilde, to_dev

pytestmark = pytest.mark.gpu

R, PAGE, ROW = 512, 64, 288


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


def _rows(shape, seed, std=1.0):
    """bf16 bits of rows whose channels have unlike spread."""
    x = oracle.widen(synth.normal_bf16(tuple(shape) + (R,), seed, synth.STREAM_CACHE, std))
    gain = np.exp2(np.arange(R) % 7 - 3.0)
    return synth.f64_to_bf16_bits(x * gain)


def _setup(lens, room, seed, unit=1.0, fill=0xA7):
    """A pool whose unused rows hold `fill` bytes (0xA7 is a code pair and a tiny scale; 0x7F a
    NaN scale), tables that map ceil((L + room) / 64) pages, and the float64 rows."""
    lens = np.asarray(lens, dtype=np.int32)
    table, P = synth.page_layout(lens + room, seed)
    pool = np.full((P, PAGE, ROW), fill, dtype=np.uint8)
    rows = oracle.widen(_rows((len(lens), max(int(lens.max()), 1)), seed))
    values = []
    for b, L in enumerate(lens):
        p = oracle.packed_quantise(rows[b, :L] * unit, unit)
        for j in range(L):
            pool[table[b, j // PAGE], j % PAGE] = p[j]
        values.append(oracle.packed_values(p, unit))
    return lens, table, pool, values


def _check(lens, values, qt_bits, window, sinks, o, lse, scale=1.0 / 16.0):
    """|o - ref| <= 2^-8 |ref| (the bf16 result) + (2^-11 + 2^-13) sum a|c|: P is rounded to fp16
    (2^-11 of each weight); a score is a sum of 512 products in fp32, at most 32 accumulations of
    partial sums below 2^7 that lose 2^-23 each, times the scale 2^-4: 2^-15.  With the
    exponential's 2^-21 a weight and the row sum each move by less than 2^-14.  A weight is held as
    2^7 p, where the largest p of a head is at least 1 (the running maximum never exceeds the
    true one): below fp16's normal range it is rounded by at most 2^-25, which over a sum of at
    least 2^7 is 2^-32 of every |c|."""
    qt = oracle.widen(qt_bits)
    o, lse = bf16_to_f64(o), lse.cpu().numpy().astype(np.float64)
    for b, L in enumerate(lens):
        for i in range(qt.shape[1]):
            at = oracle.window_positions(int(L), qt.shape[1], i, window, sinks)
            ref, ref_lse, mag = oracle.attend_rows(qt[b, i], values[b][at], scale)
            assert np.isfinite(o[b, i]).all(), (b, i, L)
            low = np.abs(values[b][at]).sum(axis=0) * 2.0 ** -32
            err = np.abs(o[b, i] - ref) - (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * mag + low)
            assert err.max() <= 1e-30, (b, i, L, window, sinks, err.max(), np.unravel_index(err.argmax(), err.shape))
            if at.size == 0:
                assert np.isneginf(lse[b, i]).all()
            else:
                # a weighted mean of score errors, and log2 / exp2 in fp32
                assert np.abs(lse[b, i] - ref_lse).max() <= 2.0 ** -14 + 2.0 ** -22 * np.abs(ref_lse).max()


LENS = [1, 300, 64, 65, 127, 128, 129, 63, 257, 1000, 2]


@pytest.mark.parametrize("unit", [1.0, 0.125, 64.0])
@pytest.mark.parametrize("q_len", [1, 6, 64, 65, 200])
def test_append_matches_oracle_bitwise(unit, q_len):
    lens0 = np.array([0, 1, 63, 64, 100], dtype=np.int32)
    lens, table, pool, _ = _setup(lens0, q_len, seed=1, unit=unit)
    rows = _rows((len(lens), q_len), 7, std=unit)
    flat = rows.reshape(-1)
    flat[:8] = synth.f64_to_bf16_bits(np.array([0.0, -0.0, 1e-30, -3e38, 3e38, 1e-5, 448.0, 2.0]))
    rows[1, 0, 16:32] = 0                                 # a zero group
    rows[2, 0, 40] = 0x7F80                               # Inf
    rows[3, 0, 511] = 0x7FC0                              # NaN
    rows[4, 0, :16] = synth.f64_to_bf16_bits(np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5,
                                                       -3.5, -5, -6]) * unit)  # ties
    d_pool, d_lens, st = torch.from_numpy(pool).cuda(), ints_to_dev(lens), _status()
    m.mla_cache_append_packed(d_pool, ints_to_dev(table), d_lens, to_dev(rows), unit=unit, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert d_lens.cpu().numpy().tolist() == (lens + q_len).tolist()
    want = pool.copy()
    packed = oracle.packed_quantise(oracle.widen(rows), unit)
    for b in range(len(lens)):
        for i in range(q_len):
            j = int(lens[b]) + i
            want[table[b, j // PAGE], j % PAGE] = packed[b, i]
    got = d_pool.cpu().numpy()
    bad = np.argwhere(got != want)
    assert bad.size == 0, (bad[:5], got[tuple(bad[0])], want[tuple(bad[0])])
    back = m.mla_cache_unpack(d_pool, ints_to_dev(table), ints_to_dev(lens), q_len, unit=unit, status=st)
    ref = oracle.packed_values(packed, unit)
    got = bf16_to_f64(back)
    assert int(st.item()) == 0
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])


def test_append_and_unpack_errors_leave_the_sequence():
    table = np.array([[0, -1], [1, 2], [3, 9]], dtype=np.int32)
    pool = np.full((4, PAGE, ROW), 5, dtype=np.uint8)
    for q_len in (6, 65):
        lens = np.array([60, 10, 63], dtype=np.int32)
        d_pool, d_lens, st = torch.from_numpy(pool).cuda(), ints_to_dev(lens), _status()
        rows = _rows((3, q_len), 3)
        m.mla_cache_append_packed(d_pool, ints_to_dev(table), d_lens, to_dev(rows), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == m.MLA_ERR_INDEX
        assert d_lens.cpu().numpy().tolist() == [60, 10 + q_len, 63]
        got = d_pool.cpu().numpy()
        assert (got[0] == 5).all() and (got[3] == 5).all()
        assert np.array_equal(got[1, 10:10 + min(q_len, 54)], oracle.packed_quantise(oracle.widen(rows))[1, :54])
    st = _status()
    back = m.mla_cache_unpack(d_pool, ints_to_dev(table), ints_to_dev([62, 0, -1]), 3, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == m.MLA_ERR_INDEX
    back = bf16_to_f64(back)
    assert back[0, :2].any(axis=-1).all() and not back[0, 2].any() and not back[2].any()


def test_truncate_matches_bf16_semantics():
    q_len = 6
    lens, table, pool, _ = _setup([6, 64, 70, 130], 0, seed=2)
    keep = np.array([0, 6, 3, 1], dtype=np.int32)
    d_pool, d_lens, st = torch.from_numpy(pool).cuda(), ints_to_dev(lens), _status()
    m.mla_cache_truncate_packed(d_pool, ints_to_dev(table), d_lens, ints_to_dev(keep), q_len, status=st)
    torch.cuda.synchronize()
    want = pool.copy()
    for b in range(4):
        for j in range(int(lens[b]) - q_len + int(keep[b]), int(lens[b])):
            want[table[b, j // PAGE], j % PAGE] = 0
    assert int(st.item()) == 0
    assert np.array_equal(d_pool.cpu().numpy(), want)
    assert d_lens.cpu().numpy().tolist() == (lens - q_len + keep).tolist()
    m.mla_cache_truncate_packed(d_pool, ints_to_dev(table), d_lens, ints_to_dev([7, -1, 0, 0]), q_len, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == m.MLA_ERR_INDEX and d_lens.cpu().numpy().tolist() == [0, 64, 61, 119]


@pytest.mark.parametrize("fill", [0xA7, 0x7F, 0xFF])
@pytest.mark.parametrize("q_len", [1, 2, 6])
def test_attend_matches_float64(q_len, fill):
    lens, table, pool, values = _setup([max(L, q_len) for L in LENS], 0, seed=3, fill=fill)
    qt = synthetic_qtilde(len(lens), q_len, seed=4)
    st = _status()
    o, lse = m.mla_attend_packed(to_dev(qt), torch.from_numpy(pool).cuda(), ints_to_dev(table), ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _check(lens, values, qt, 0, 0, o, lse)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (100, 5), (128, 64), (129, 130), (500, 0), (4000, 3), (1, 700)])
@pytest.mark.parametrize("q_len", [1, 6])
def test_attend_windows(window, sinks, q_len):
    """Rows outside every query's window hold NaN scales and their pages may be unmapped."""
    lens, table, pool, values = _setup([max(L, q_len) for L in LENS], 0, seed=5, fill=0x7F)
    for b, L in enumerate(lens):
        seen = np.zeros(int(L), dtype=bool)
        for i in range(q_len):
            seen[oracle.window_positions(int(L), q_len, i, window, sinks)] = True
        for j in np.flatnonzero(~seen):
            pool[table[b, j // PAGE], j % PAGE] = 0x7F
        for pg in range(-(-int(L) // PAGE)):
            if not seen[pg * PAGE:(pg + 1) * PAGE].any():
                table[b, pg] = -1 if pg % 2 else 1 << 30
    qt = synthetic_qtilde(len(lens), q_len, seed=6)
    st = _status()
    o, lse = m.mla_attend_packed(to_dev(qt), torch.from_numpy(pool).cuda(), ints_to_dev(table), ints_to_dev(lens),
                                 window=window, sinks=sinks, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _check(lens, values, qt, window, sinks, o, lse)


def test_attend_empty_rows_units_and_scales():
    """Sequences shorter than the query window (some queries see nothing), a unit, a scale."""
    lens, table, pool, values = _setup([0, 1, 3, 200, 0, 5], 0, seed=8, unit=0.25)
    qt = synthetic_qtilde(len(lens), 6, seed=9)
    st = _status()
    o, lse = m.mla_attend_packed(to_dev(qt), torch.from_numpy(pool).cuda(), ints_to_dev(table), ints_to_dev(lens),
                                 unit=0.25, scale=0.03, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _check(lens, values, qt, 0, 0, o, lse, scale=0.03)
    none, _, pool0, _ = _setup([0, 0], 64, seed=8)
    o, lse = m.mla_attend_packed(to_dev(qt[:2]), torch.from_numpy(pool0).cuda(), ints_to_dev(table[:2]), ints_to_dev(none),
                                 status=st)
    assert not o.float().any() and torch.isneginf(lse).all() and int(st.item()) == 0


@pytest.mark.parametrize("spread", [1e-20, 1.0, 1e20])
def test_attend_query_ranges_and_rising_scores(spread):
    """Heads of very unlike size, scores that rise along the sequence (every tile raises the
    running maximum, so O is rescaled in tensor memory), and one zero head."""
    lens, table, pool, _ = _setup([900], 0, seed=10)
    qt = oracle.widen(synthetic_qtilde(1, 1, seed=11))
    qt *= np.exp2(np.arange(64) % 9 - 4.0)[None, None, :, None]
    qt[0, 0, 5] = 0
    rows = oracle.widen(_rows((900,), 12))
    rows += (np.arange(900) / 150.0)[:, None] * np.sign(qt[0, 0, 3])[None]
    p = oracle.packed_quantise(rows)
    for j in range(900):
        pool[table[0, j // PAGE], j % PAGE] = p[j]
    bits = synth.f64_to_bf16_bits(qt * spread)
    st = _status()
    scale = float(np.float32(1.0 / 16.0 / spread))
    o, lse = m.mla_attend_packed(to_dev(bits), torch.from_numpy(pool).cuda(), ints_to_dev(table), ints_to_dev(lens),
                                 scale=scale, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    v = oracle.packed_values(p)
    ref, ref_lse, mag = oracle.attend_rows(oracle.widen(bits)[0, 0], v, scale)
    # scores reach some 2^9 here (partial sums before the scale 2^13): 32 accumulations of 2^-23
    # of that, times 2^-4, are 2^-9 of a weight in the worst case
    s = np.abs(oracle.widen(bits)[0, 0]) @ np.abs(v).T * scale
    rel = 2.0 ** -11 + 2 * s.max(axis=1, keepdims=True) * 32 * 2.0 ** -23
    err = np.abs(bf16_to_f64(o)[0, 0] - ref) - (2.0 ** -8 * np.abs(ref) + rel * mag + np.abs(v).sum(axis=0) * 2.0 ** -32)
    assert err.max() <= 1e-30
    assert (np.abs(lse.cpu().numpy()[0, 0] - ref_lse) <= rel[:, 0] + 2.0 ** -22 * np.abs(ref_lse)).all()


def test_attend_nan_rows_show_and_bad_pages_are_flagged():
    lens, table, pool, values = _setup([200, 200], 0, seed=13)
    pool[table[0, 1], 3, 256 + 7] = 0x7F  # group 7 of position 67 of sequence 0
    qt = synthetic_qtilde(2, 1, seed=14)
    st = _status()
    args = (to_dev(qt), torch.from_numpy(pool).cuda())
    o, lse = m.mla_attend_packed(*args, ints_to_dev(table), ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.isnan(o[0].float()).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(o[1].float()).all() and torch.isfinite(lse[1]).all()
    for bad in (-1, pool.shape[0], 1 << 30):
        t2 = table.copy()
        t2[1, 2] = bad
        st.zero_()
        m.mla_attend_packed(*args, ints_to_dev(t2), ints_to_dev(lens), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == m.MLA_ERR_INDEX
    st.zero_()
    m.mla_attend_packed(*args, ints_to_dev(table), ints_to_dev([200, table.shape[1] * 64 + 1]), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == m.MLA_ERR_INDEX


def test_attend_many_queries_and_many_sequences():
    """More queries than SMs (a prefill through this path), and more sequences than SMs."""
    for lens, q_len, window, sinks in (([300], 300, 0, 0), ([300], 200, 70, 3), ([90 + 5 * b for b in range(200)], 1, 0, 0)):
        lens, table, pool, values = _setup(lens, 0, seed=15)
        qt = synthetic_qtilde(len(lens), q_len, seed=16)
        st = _status()
        o, lse = m.mla_attend_packed(to_dev(qt), torch.from_numpy(pool).cuda(), ints_to_dev(table), ints_to_dev(lens),
                                     window=window, sinks=sinks, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        _check(lens, values, qt, window, sinks, o, lse)


# a single row, some sequences with many partials, with few, and more sequences than CTA groups
MERGES = [(1, [0]), (1, [1]), (1, [300]), (1, [18944]), (1, [20001]), (2, [5000]), (6, [4100]), (1, [8000, 37]), (1, [0, 6000, 3]),
          (1, [700] * 9), (1, [1200 + 77 * k for k in range(12)]), (8, [118] * 25), (8, [9 + 13 * k for k in range(20)]),
          (1, [100] * 148), (1, [k % 5 * 130 for k in range(160)])]


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
@pytest.mark.parametrize("q_len,lens", MERGES, ids=[f"{len(x)}x{q}x{max(x)}" for q, x in MERGES])
def test_merges_read_only_what_the_call_wrote(q_len, lens, window, sinks):
    """The workspace holds NaN before the call; twice, with the first call's contents before the second."""
    room = 0 if max(lens) else 1  # a pool and a table have at least one page (no pages: MLA_ERR_ARG)
    lens, table, pool, values = _setup(lens, room, seed=31)
    qt = synthetic_qtilde(len(lens), q_len, seed=32)
    ws = m.new_workspace(len(lens), q_len)
    ws.fill_(0xFF)
    st = _status()
    args = (to_dev(qt), torch.from_numpy(pool).cuda(), ints_to_dev(table), ints_to_dev(lens))
    o, lse = m.mla_attend_packed(*args, window=window, sinks=sinks, workspace=ws, status=st)
    again, lse_again = m.mla_attend_packed(*args, window=window, sinks=sinks, workspace=ws, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(o, again) and torch.equal(lse, lse_again)
    _check(lens, values, qt, window, sinks, o, lse)


# Every form of the merge, a tile per CTA: a single row; few sequences; more; as many as CTA groups.
TILE_EACH = [[12801], [6401, 6400], [257] * 20, [257] * 40 + [0] * 110]


@pytest.mark.parametrize("what", ["query", "row", "last row"])
@pytest.mark.parametrize("lens", TILE_EACH, ids=[f"{len(x)}x{max(x)}" for x in TILE_EACH])
def test_nan_shows_whatever_its_weight(lens, what):
    """Head 0 of every sequence scores 200 and more at row 3 and about 0 elsewhere: the other tiles'
    partials have the weight 2^-288 or less, zero in fp32, and a NaN in them still counts (0 x NaN)."""
    lens, table, pool, _ = _setup(lens, 0, seed=40)
    qt = synthetic_qtilde(len(lens), 1, seed=41)
    q = oracle.widen(qt)[:, 0, 0]
    assert np.abs(q).sum(axis=1).min() > 200
    pool[..., 256:] = 0x01  # scales of 2^-9
    high = oracle.packed_quantise(np.sign(q) * 16.0)
    for b in np.flatnonzero(lens):
        pool[table[b, 0], 3] = high[b]
    if what == "query":
        qt[0, 0, 5, 100] = 0x7FC0
    else:
        j = int(lens[0]) - 1 if what == "last row" else 200
        pool[table[0, j // PAGE], j % PAGE, 256 + 7] = 0x7F
    st = _status()
    o, lse = m.mla_attend_packed(to_dev(qt), torch.from_numpy(pool).cuda(), ints_to_dev(table), ints_to_dev(lens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    bad = [5] if what == "query" else list(range(64))
    fine = [h for h in range(64) if h not in bad]
    assert torch.isnan(o[0, 0, bad]).all() and torch.isnan(lse[0, 0, bad]).all()
    assert torch.isfinite(o[0, 0, fine].float()).all() and torch.isfinite(lse[0, 0, fine]).all()
    assert torch.isfinite(o[1:].float()).all() and torch.isfinite(lse[1:][ints_to_dev(lens[1:]) > 0]).all()
