"""csa2_page_tables against a Python model: growth, drops, pages handed on within a call, kept pages,
padding rows, refusals that change nothing, in-place steps replayed from a graph."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from paged_common import PagedState

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def i32(v):
    return to_dev(np.asarray(v, np.int32))


class Device:
    """Device arrays of one model state."""

    def __init__(self, s, n_rows):
        self.have, self.table = i32(s.have), i32(s.table)
        self.free, self.n_free = i32(s.free), i32([s.n_free])
        e = lambda n, t: torch.full((max(n, 1),), -77, dtype=t, device="cuda")
        self.n_entries, self.n_free_out, self.row_start = e(s.B, torch.int32), e(1, torch.int32), e(s.B + 1, torch.int32)
        self.query, self.slot = e(n_rows, torch.int32), e(n_rows, torch.int32)
        self.entry, self.pos = e(n_rows, torch.int64), e(n_rows, torch.int64)
        self.n_rows = n_rows
        self.ws = csa2.workspace(csa2.page_tables_workspace_size(s.B))

    def call(self, s, new, kept, m, inplace=False):
        csa2.page_tables(s.B, self.have, new, s.P, self.table, s.max_pages, s.n_pages, self.free, self.n_free,
                         self.n_free if inplace else self.n_free_out, self.have if inplace else self.n_entries,
                         self.ws, n_rows=self.n_rows, query=self.query if self.n_rows else None,
                         slot=self.slot if self.n_rows else None, entry=self.entry if self.n_rows else None,
                         pos=self.pos if self.n_rows else None, row_start=self.row_start, m=m, n_kept=kept)


def check(d, s, rows, start, n_rows, inplace=False):
    host = lambda t: t.cpu().numpy()
    assert np.array_equal(host(d.table), np.array(s.table, np.int32))
    assert np.array_equal(host(d.free), np.array(s.free, np.int32))
    assert host(d.n_free if inplace else d.n_free_out)[0] == s.n_free
    assert np.array_equal(host(d.have if inplace else d.n_entries), s.have)
    assert np.array_equal(host(d.row_start), start)
    if n_rows:
        want = np.full((n_rows, 4), -1, np.int64)
        if rows:
            want[:len(rows)] = rows
        got = np.stack([host(d.query), host(d.slot), host(d.entry), host(d.pos)], 1)
        assert np.array_equal(got, want)


def fresh(rng, B, P, max_pages, spare, have_max):
    have = [int(rng.integers(0, have_max + 1)) for _ in range(B)]
    used = sum(-(-h // P) for h in have)
    ids = [int(x) for x in rng.permutation(used + spare)]
    s = PagedState(B, P, max_pages, used + spare, ids[used:])
    at = 0
    for b in range(B):
        s.have[b] = have[b]
        for p in range(-(-have[b] // P)):
            s.table[b][p] = ids[at]
            at += 1
    return s


@pytest.mark.parametrize("B,P,have,new,pad,m,drops", [
    (1, 1, 0, 1, 0, 1, False), (1, 64, 63, 1, 2, 128, False), (3, 7, 50, 30, 1, 2, True), (32, 16, 200, 1, 5, 1, False),
    (33, 16, 200, 20, 0, 4, True), (1025, 8, 40, 9, 3, 1, True), (2048, 3, 9, 3, 1, 1, True),
    (2049, 5, 9, 3, 4, 1, True),          # beyond one CTA's requests
    (7, 64, 1000, 4000, 9, 128, True),    # beyond one CTA's rows
    (300, 1, 40, 40, 0, 1, True),         # thousands of pages change hands in one CTA
    (65535, 16, 40, 2, 0, 1, True)])
def test_tables_match_the_model(B, P, have, new, pad, m, drops):
    rng = np.random.default_rng(B * 131 + P)
    max_pages = -(-(have + 4 * new) // P) + 1
    s = fresh(rng, B, P, max_pages, 2 + B * 2 * (-(-new // P)), have)
    for _ in range(2):  # two steps, each from the last one's state
        add = [int(rng.integers(-min(new, s.have[b]) if drops else 0, new + 1)) for b in range(B)]
        if drops and B > 2:
            add[1] = -s.have[1]
        kept = [int(rng.integers(0, 3)) for _ in range(B)]
        n_rows = sum(max(a, 0) for a in add) + pad
        d = Device(s, n_rows)
        rows, start = s.step(add, kept, m, n_rows)
        assert rows != 6 and rows != 7
        d.call_new = i32(add)
        d.call(s, d.call_new, i32(kept), m)
        assert csa2.check(d.ws)[0] == 0
        check(d, s, rows, start, n_rows)
        d.call(s, d.call_new, i32(kept), m)  # the inputs are as they were: once more gives the same
        check(d, s, rows, start, n_rows)


def test_lengths_without_maps_and_without_kept():
    rng = np.random.default_rng(3)
    s = fresh(rng, 6, 4, 12, 20, 20)
    d = Device(s, 0)
    add = [1, 0, 9, -3, 0, 4]
    add[3] = -min(3, s.have[3])
    rows, start = s.step(add, [0] * 6, 1, None)
    csa2.page_tables(6, d.have, i32(add), 4, d.table, 12, s.n_pages, d.free, d.n_free, d.n_free_out, d.n_entries, d.ws)
    assert csa2.check(d.ws)[0] == 0
    d.row_start = i32(start)
    check(d, s, rows, start, 0)


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("fault,status", [("short", 7), ("rows", 6), ("negative", 6), ("long", 6), ("stack", 6),
                                          ("free id", 6), ("table id", 6), ("n_free", 6), ("kept", 6), ("have", 6)])
def test_refused_call_changes_nothing(fault, status, big):
    rng = np.random.default_rng(5)
    B, P = (2100 if big else 9), 4
    s = fresh(rng, B, P, 16, 3 * B, 20)
    add = [int(rng.integers(0, 5)) for _ in range(B)]
    kept = [0] * B
    if s.have[2] < 8:  # a request to drop from
        add[2] = 8
        s.step(add, kept, 1, None)
    add = [1] * B
    add[2] = -s.have[2]
    n_rows = B
    detail = None
    if fault == "short":
        add = [P] * B  # a page each
        add[2] = -s.have[2]
        n_rows, need, back = P * B, B - 1, -(-s.have[2] // P)
        assert need > back
        s.n_free = need - back - 1
        detail = 1
    elif fault == "rows":
        n_rows, detail = B - 2, B - 1
    elif fault == "negative":
        add[4], detail = -s.have[4] - 1, 4
    elif fault == "long":
        add[5], detail = 16 * P + 1, 5
    elif fault == "stack":
        s.n_free = s.n_pages
        s.free = [0] * s.n_pages
    elif fault == "free id":
        for i in range(s.n_free):
            s.free[i] = s.n_pages
        add = [P] * B
        n_rows, detail = P * B, s.n_pages
    elif fault == "table id":
        s.table[2][0], detail = -5, -5
    elif fault == "n_free":
        s.n_free = detail = s.n_pages + 1
    elif fault == "kept":
        kept[3], detail = -1, 3
    elif fault == "have":
        s.have[6], detail = -2, 6
    d = Device(s, n_rows)
    d.call(s, i32(add), i32(kept), 1)
    st, det = csa2.check(d.ws)
    assert st == status
    if detail is not None:
        assert det == detail
    check(d, s, [], [0] * (B + 1), n_rows)


def test_no_pages_detail_and_pages_handed_on():
    # request 0 ends and gives its three pages to requests 1 and 2 in the same call; one more is missing
    s = PagedState(3, 2, 8, 8, [])
    s.have = [6, 2, 2]
    s.table[0][:3], s.table[1][0], s.table[2][0] = [4, 5, 6], 0, 1
    d = Device(s, 8)
    d.call(s, i32([-6, 4, 3]), None, 1)  # needs 2 + 2 pages, 3 come back
    assert csa2.check(d.ws) == (7, 1)
    check(d, s, [], [0] * 4, 8)
    add = [-6, 4, 2]
    rows, start = s.step(add, [0] * 3, 1, 8)
    d.call(s, i32(add), None, 1)
    assert csa2.check(d.ws)[0] == 0
    check(d, s, rows, start, 8)
    assert sorted(s.table[1][1:3] + s.table[2][1:2]) == [4, 5, 6] and s.n_free == 0


@pytest.mark.parametrize("B", [40, 2100])
def test_steps_in_place_from_a_graph_on_another_stream(B):
    rng = np.random.default_rng(11)
    P = 16
    s = fresh(rng, B, P, 20, 5 * B, 100)  # 38 entries more need three pages each at most
    d = Device(s, B)
    add, kept = [1] * B, [0] * B
    new = i32(add)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        d.call(s, new, None, 1, inplace=True)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            d.call(s, new, None, 1, inplace=True)
        rows, start = s.step(add, kept, 1, B)  # the warm call; the captured one has not run
        for _ in range(37):
            g.replay()
            rows, start = s.step(add, kept, 1, B)
    st.synchronize()
    assert csa2.check(d.ws)[0] == 0
    check(d, s, rows, start, B, inplace=True)


@pytest.mark.parametrize("table", [None, torch.empty((3, 0), dtype=torch.int32)])
def test_no_request_has_or_gets_an_entry(table):
    table = table if table is None else table.cuda()
    e = lambda *n: torch.full(n, -77, dtype=torch.int32, device="cuda")
    free, n_free, n_free_out, n_entries, start, query = i32([4, 2, 9]), i32([3]), e(1), e(3), e(4), e(5)
    ws = csa2.workspace(csa2.page_tables_workspace_size(3))
    call = lambda new: csa2.page_tables(3, i32([0, 0, 0]), i32(new), 16, table, 0, 10, free, n_free, n_free_out, n_entries,
                                        ws, n_rows=5, query=query, row_start=start)
    call([0, 0, 0])
    assert csa2.check(ws)[0] == 0
    assert n_entries.tolist() == [0, 0, 0] and n_free_out.tolist() == [3] and start.tolist() == [0] * 4
    assert query.tolist() == [-1] * 5 and free.tolist() == [4, 2, 9]
    call([0, 1, 0])
    assert csa2.check(ws) == (6, 1)
    assert n_entries.tolist() == [0, 0, 0] and n_free_out.tolist() == [3]
