"""Page bookkeeping on the GPU against the one-entry-at-a-time oracle, bit for bit: tables, counts,
lengths and every byte of the pool."""
import numpy as np
import pytest
import torch

import mla_absorbed_latent_mtp_b200 as m
import oracle
from gpu_util import ints_to_dev

pytestmark = pytest.mark.gpu

PAGE = 64
CODES = {"ok": 0, "index": m.MLA_ERR_INDEX, "pages": m.MLA_ERR_PAGES}


@pytest.fixture(scope="module", autouse=True)
def device():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


class Both:
    """The same state on the GPU and in the oracle; call() runs an operation on both and compares."""

    def __init__(self, table, lens, refs, pool):
        self.book = oracle.PageBook(table.copy(), lens.copy(), refs.copy(), pool.copy())
        self.table, self.lens, self.refs = ints_to_dev(table), ints_to_dev(lens), ints_to_dev(refs)
        self.pool = torch.from_numpy(pool).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, name, *args):
        self.status.zero_()
        a = [ints_to_dev(x) if isinstance(x, (list, np.ndarray)) else x for x in args]
        got = None
        if name == "reserve":
            m.mla_pages_reserve(self.pool, self.table, self.lens, self.refs, *a, status=self.status)
        elif name == "fork":
            m.mla_pages_fork(self.pool, self.table, self.lens, self.refs, *a, status=self.status)
        elif name == "release":
            m.mla_pages_release(self.table, self.lens, self.refs, status=self.status)
        else:
            got = m.mla_pages_compact(self.pool, self.table, self.refs, status=self.status)
        torch.cuda.synchronize()
        want = getattr(self.book, name)(*args)
        if name == "compact":
            assert int(got.item()) == want
            want = "ok"
        assert int(self.status.item()) == CODES[want] or \
            (want != "ok" and int(self.status.item()) in (m.MLA_ERR_INDEX, m.MLA_ERR_PAGES)), (name, args)
        assert np.array_equal(self.table.cpu().numpy(), self.book.table), name
        assert np.array_equal(self.lens.cpu().numpy(), self.book.lens), name
        assert np.array_equal(self.refs.cpu().numpy(), self.book.refs), name
        assert np.array_equal(self.pool.cpu().numpy(), self.book.pool), name
        # the counts are the table's
        mapped = self.book.table[self.book.table >= 0]
        mapped = mapped[mapped < len(self.book.refs)]
        assert np.array_equal(np.bincount(mapped, minlength=len(self.book.refs)), self.book.refs)
        return want


def _state(rng, B, lens, max_pages, P, width=288):
    table = np.full((B, max_pages), -1, dtype=np.int32)
    free = list(rng.permutation(P))
    for b in range(B):
        for k in range(-(-int(lens[b]) // PAGE)):
            table[b, k] = free.pop()
    refs = np.bincount(table[table >= 0], minlength=P).astype(np.int32)
    pool = rng.integers(0, 256, (P, PAGE, width), dtype=np.uint8)
    return Both(table, np.asarray(lens, dtype=np.int32), refs, pool)


@pytest.mark.parametrize("width", [16, 48, 288, 1024])
def test_a_life_of_a_cache(width):
    """Reserve, append (the lengths move), fork, diverge, truncate, release, compact, again."""
    rng = np.random.default_rng(width)
    B, max_pages, P = 9, 6, 40
    lens = [0, 1, 63, 64, 65, 128, 200, 0, 0]
    s = _state(rng, B, lens, max_pages, P, width)
    for step in range(3):
        s.call("reserve", 6)
        for b in range(7):  # the appends
            s.book.lens[b] += 6
        s.lens += ints_to_dev([6] * 7 + [0, 0])
        s.call("fork", [2, 6], [7, 8])
        s.call("reserve", 70)
        s.book.lens[1::2] += 70
        s.lens[1::2] += 70
        s.book.lens[3] -= 66
        s.lens[3] -= 66
        s.call("release")
        s.call("compact")
        for b in (7, 8):
            s.book.lens[b] = 0
            s.lens[b] = 0
        s.call("release")
        if step == 1:
            s.call("compact")
        for b in range(7):
            cut = min(int(s.book.lens[b]), 70)
            s.book.lens[b] -= cut
            s.lens[b] -= cut


def test_shared_pages_are_copied_before_they_are_written():
    rng = np.random.default_rng(1)
    s = _state(rng, 4, [130, 64, 0, 0], 4, 20)
    s.call("fork", [0, 0], [2, 3])          # three sequences share two full pages
    for b in (0, 2):                        # two of them go back into a shared page
        s.book.lens[b] = 70
        s.lens[b] = 70
    assert s.call("reserve", 3) == "ok"
    assert s.book.table[0, 1] != s.book.table[2, 1] and s.book.table[3, 1] not in (s.book.table[0, 1], s.book.table[2, 1])
    assert s.book.refs[s.book.table[3, 1]] == 1 and s.book.refs[s.book.table[3, 0]] == 3
    s.call("reserve", 3)                    # nothing is shared there any more
    s.call("release")
    s.call("compact")


def test_pages_run_out_in_order():
    rng = np.random.default_rng(2)
    s = _state(rng, 6, [64, 64, 10, 64, 64, 64], 4, 8)  # six mapped, two free
    assert s.call("reserve", 1) == "pages"              # sequences 0 and 1 get them, 2 needs none
    assert [int((r >= 0).sum()) for r in s.book.table] == [2, 2, 1, 1, 1, 1]
    s = _state(rng, 5, [70, 70, 0, 0, 0], 4, 5)
    assert s.call("fork", [0, 1, 0], [2, 3, 4]) == "pages"
    assert s.book.lens.tolist() == [70, 70, 70, 0, 0]


def test_refused_entries_are_left_alone():
    rng = np.random.default_rng(3)
    s = _state(rng, 8, [130, 64, 5, 0, 0, 0, 0, 0], 4, 30)
    # parent or child out of range, itself, a child twice, a child that is a parent, a full child
    assert s.call("fork", [0, -1, 8, 1, 0, 1, 5, 0, 0], [3, 4, 5, 1, 6, 6, 7, 9, 2]) == "index"
    assert s.book.lens.tolist() == [130, 64, 5, 130, 0, 0, 0, 0]
    s = _state(rng, 3, [250, 10, 3], 4, 30)
    assert s.call("reserve", 7) == "index"  # 257 rows do not fit four pages
    assert (s.book.table[0] >= 0).sum() == 4 and (s.book.table[1] >= 0).sum() == 1
    s.book.lens[1] = -3
    s.lens[1] = -3
    assert s.call("reserve", 1) == "index"
    assert s.call("release") == "index"


def test_bad_table_entries_are_flagged():
    rng = np.random.default_rng(4)
    for bad in (-2, 30, 1 << 30):
        s = _state(rng, 3, [130, 64, 5], 4, 30)
        s.book.table[0, 2] = bad
        s.book.refs[:] = np.bincount(s.book.table[(s.book.table >= 0) & (s.book.table < 30)], minlength=30)
        s.table.copy_(ints_to_dev(s.book.table))
        s.refs.copy_(ints_to_dev(s.book.refs))
        assert s.call("reserve", 1) == "index"
        s.book.lens[0] = 100
        s.lens[0] = 100
        assert s.call("release") == "index"
        m.mla_pages_compact(s.pool, s.table, s.refs, status=s.status)
        torch.cuda.synchronize()
        assert int(s.status.item()) == m.MLA_ERR_INDEX and int(s.table[0, 2].item()) == bad


@pytest.mark.parametrize("P", [1, 31, 33, 4095, 4096, 4097, 12300])
def test_pool_sizes_around_the_snapshot_chunks(P):
    rng = np.random.default_rng(P)
    B = min(40, P)
    each = max(1, P // (2 * B))
    lens = rng.integers(0, each * PAGE + 1, B)
    s = _state(rng, B, lens, each + 2, P, 16)
    s.call("reserve", 65)
    s.call("compact")
    s.book.lens[: B // 2] = 0
    s.lens[: B // 2] = 0
    s.call("release")
    s.call("compact")
    if B >= 8:
        s.call("fork", list(range(B // 2, B // 2 + 4)), [0, 1, 2, 3])


def test_full_and_empty_pools():
    rng = np.random.default_rng(5)
    s = _state(rng, 2, [128, 128], 3, 4)
    s.call("compact")
    assert s.call("reserve", 1) == "pages"
    s.book.lens[:] = 0
    s.lens.zero_()
    s.call("release")
    s.call("compact")
    assert s.call("reserve", 192) == "pages"


def test_bf16_pool_and_attention_after_a_fork_and_a_compaction():
    """The pages move, the rows a sequence attends do not: results before and after are the same bits."""
    rng = np.random.default_rng(6)
    lens = [200, 70, 0, 129]
    B, max_pages, P = 4, 5, 24
    s = _state(rng, B, lens, max_pages, P, 1024)
    pool = torch.randn(P, PAGE, 512, device="cuda", dtype=torch.bfloat16)
    qt = torch.randn(B, 1, 64, 512, device="cuda", dtype=torch.bfloat16)
    before, _ = m.mla_attend_paged(qt, pool, s.table, s.lens)
    m.mla_pages_fork(pool, s.table, s.lens, s.refs, ints_to_dev([0]), ints_to_dev([2]), status=s.status)
    m.mla_pages_compact(pool, s.table, s.refs, status=s.status)
    qt[2] = qt[0]
    after, _ = m.mla_attend_paged(qt, pool, s.table, s.lens)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    assert torch.equal(after[[0, 1, 3]], before[[0, 1, 3]])
    # the fork attends the same rows (the split of the tile list differs: rounding may)
    assert (after[2].float() - before[0].float()).abs().max() <= 2.0 ** -7 * before[0].float().abs().max()
    # the child's copy is its own
    assert int(s.table[2, 3].item()) != int(s.table[0, 3].item()) and torch.equal(s.table[2, :3], s.table[0, :3])


def test_demands_past_32_bits():
    """66 sequences that ask for 2^25 - 1 pages each: their sum passes 2^31, none has room, and
    nothing changes."""
    B, max_pages, P = 66, 2 ** 25 - 1, 64
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    pool = torch.zeros(P, PAGE, 16, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.mla_pages_reserve(pool, table, lens, refs, max_pages * PAGE, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == m.MLA_ERR_PAGES
    assert int(refs.abs().max().item()) == 0
    assert int(table.amax().item()) == -1 and int(table.amin().item()) == -1


@pytest.mark.parametrize("low", [True, False])
def test_compaction_flags_entries_that_map_free_pages(low):
    """Below and above the pages in use: the entry stays, the status says so."""
    refs = torch.ones(10, dtype=torch.int32, device="cuda")
    page = 1 if low else 9
    refs[page] = refs[2] = 0
    table = torch.tensor([[0, 3, 4, 5], [6, 7, 8, page], [9 if low else 1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    pool = torch.arange(10, dtype=torch.uint8, device="cuda")[:, None, None].repeat(1, PAGE, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = m.mla_pages_compact(pool, table, refs, status=status)
    torch.cuda.synchronize()
    assert int(n.item()) == 8 and int(status.item()) == m.MLA_ERR_INDEX and int(table[1, 3].item()) == page
    # used pages at or above 8 move, in order, to the free ones: low {8, 9} to {1, 2}, else {8} to {2}
    assert table[1, 2].item() == (1 if low else 2) and table[2, 0].item() == (2 if low else 1)
    assert int(pool[int(table[1, 2].item()), 0, 0].item()) == 8


def _give_back(s, b, entries):
    """What a caller does with pages that no window reaches any more."""
    for k in entries:
        s.book.refs[s.book.table[b, k]] -= 1
        s.book.table[b, k] = -1
    s.table.copy_(ints_to_dev(s.book.table))
    s.refs.copy_(ints_to_dev(s.book.refs))


def test_a_sequence_whose_early_pages_were_given_back():
    """Its fork leaves the same entries unmapped; both go on, move, and give their tails back."""
    rng = np.random.default_rng(7)
    s = _state(rng, 4, [450, 320, 0, 0], 9, 40)
    _give_back(s, 0, [1, 2, 4])
    _give_back(s, 1, [0, 1, 2, 3])
    assert s.call("fork", [0, 1], [2, 3]) == "ok"  # a partial last page, and none
    assert s.book.lens.tolist() == [450, 320, 450, 320]
    assert (s.book.table[2, :9] < 0).tolist() == [False, True, True, False, True, False, False, False, True]
    assert (s.book.table[3, :5] < 0).tolist() == [True] * 4 + [False]
    assert s.call("reserve", 70) == "ok"
    assert s.call("compact") == "ok"
    for b in range(4):
        s.book.lens[b] -= 70
        s.lens[b] -= 70
    assert s.call("release") == "ok"
    assert s.call("reserve", 6) == "ok"            # into pages that parent and child share


def test_a_fork_needs_the_page_it_copies():
    rng = np.random.default_rng(8)
    s = _state(rng, 3, [450, 0, 0], 9, 40)
    _give_back(s, 0, [7])                          # the partial last page
    assert s.call("fork", [0], [1]) == "index"
    s = _state(rng, 3, [450, 0, 0], 9, 40)
    for bad in (-2, 40, 1 << 30):
        s.book.table[0, 2] = bad
        s.book.refs[:] = np.bincount(s.book.table[(s.book.table >= 0) & (s.book.table < 40)], minlength=40)
        s.table.copy_(ints_to_dev(s.book.table))
        s.refs.copy_(ints_to_dev(s.book.refs))
        assert s.call("fork", [0], [1]) == "index"


@pytest.mark.parametrize("packed", [False, True])
def test_windowed_attention_of_a_fork_without_early_pages(packed):
    """Parent and child attend the same rows; the window's pages and the sink's are all that is mapped."""
    rng = np.random.default_rng(9)
    s = _state(rng, 2, [450, 0], 9, 40)
    _give_back(s, 0, [1, 2, 3, 4])                 # window 100 + sinks 4: pages 0, 5, 6, 7
    if packed:
        pool = torch.randint(0, 256, (40, PAGE, 288), dtype=torch.uint8, device="cuda")
        pool[..., 256:] = 0x38                     # scales of 1
    else:
        pool = torch.randn(40, PAGE, 512, device="cuda").to(torch.bfloat16)
    m.mla_pages_fork(pool, s.table, s.lens, s.refs, ints_to_dev([0]), ints_to_dev([1]), status=s.status)
    qt = torch.randn(1, 1, 64, 512, device="cuda").to(torch.bfloat16).repeat(2, 1, 1, 1)
    attend = m.mla_attend_packed if packed else m.mla_attend_window_paged
    o, lse = attend(qt, pool, s.table, s.lens, window=100, sinks=4, status=s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1]) and torch.isfinite(o.float()).all()


def test_two_page_operations_at_once():
    """On two streams, each with its own state and workspace."""
    def start(k):
        return _state(np.random.default_rng(20 + k), 40, [50 + 7 * b for b in range(30)] + [0] * 10, 12, 400, 256)

    def step(s, ws, n_used):
        m.mla_pages_fork(s.pool, s.table, s.lens, s.refs, kids[0], kids[1], workspace=ws, status=s.status)
        m.mla_pages_reserve(s.pool, s.table, s.lens, s.refs, 66, workspace=ws, status=s.status)
        m.mla_pages_release(s.table, s.lens, s.refs, status=s.status)
        m.mla_pages_compact(s.pool, s.table, s.refs, n_used=n_used, workspace=ws, status=s.status)

    kids = ints_to_dev(list(range(10))), ints_to_dev(list(range(30, 40)))
    n_useds = [ints_to_dev([0]) for _ in range(2)]
    both = [start(k) for k in range(2)]
    wss = [m.new_pages_workspace(40, 400) for _ in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for s, ws, n_used, st in zip(both, wss, n_useds, streams):
        with torch.cuda.stream(st):
            step(s, ws, n_used)
    torch.cuda.synchronize()
    for k, s in enumerate(both):
        assert int(s.status.item()) == 0
        s.book.fork(list(range(10)), list(range(30, 40)))
        s.book.reserve(66)
        s.book.release()
        assert int(n_useds[k].item()) == s.book.compact()
        for got, want in ((s.table, s.book.table), (s.lens, s.book.lens), (s.refs, s.book.refs), (s.pool, s.book.pool)):
            assert np.array_equal(got.cpu().numpy(), want)
