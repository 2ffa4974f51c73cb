"""csa2_paged_attn_decode and csa2_prefix_attn_decode against attention in float64, within the bound
that the kernels' roundings allow, at lengths, page sizes, groups and masks where they can go wrong;
the whole run of tables, appends, window and attention; refusals found on the device."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from paged_common import D, F8, H, attention, decode, norm_rope_q, random_entries

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def repeated(n, groups, shared, times):
    """The same lengths and groups with every group's queries `times` over: groups of few queries run every
    query by itself, those of five or more on average run in pairs."""
    out, new, at = [], [], 0
    for a, z in groups:
        out += n[at:a]
        new.append((len(out), len(out) + (z - a) * times))
        out += n[a:z] * times
        at = z
    return out + n[at:], new, shared


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


class Batch:
    """A paged cache on both sides: B sequences of n[b] entries in pages of P, groups of queries that
    share their first entries.  Every entry that no query may see has a NaN scale."""

    def __init__(self, seed, n, P, groups=(), shared=(), n_swa=0, win=False, extras=False, sink=False, spare=3, q=None):
        rng = np.random.default_rng(seed)
        self.B, self.P, self.n, self.n_swa, self.groups, self.shared = len(n), P, list(n), n_swa, groups, list(shared)
        B = self.B
        self.max_pages = max(1, max(-(-x // P) for x in n))
        # groups of five queries or more run in pairs where queries times n_shared_max reach 2^17: small
        # cases take a large bound (and rows as long, which are not read)
        self.shared_max = max([0, *shared])
        if groups and B >= 5 * len(groups) and B * self.shared_max < 1 << 17:
            self.shared_max = 65536
            self.max_pages = max(self.max_pages, -(-65536 // P))
        first, whole, part = list(range(B)), [0] * B, [0] * B
        for g, (a, z) in enumerate(groups):
            long = next((b for b in range(a, z) if n[b] >= shared[g]), max(range(a, z), key=lambda b: n[b]))
            for b in range(a, z):
                first[b] = long
                agree = min(shared[g], n[long], n[b])
                whole[b], part[b] = agree // P, agree % P
        count = sum(-(-n[b] // P) - (whole[b] if first[b] != b else 0) for b in range(B)) + spare
        ids = rng.permutation(count).astype(np.int32)
        self.n_pages = count
        self.codes, self.scales = random_entries(rng, count * P)
        seen = np.zeros(count * P, bool)
        # garbage behind the last page of a sequence is not read
        table = np.full((B, self.max_pages), 0x7fffffff, np.int32)
        at = 0
        self.rows = [None] * B
        for b in sorted(range(B), key=lambda b: first[b] != b):
            np_b, skip = -(-n[b] // P), whole[b] if first[b] != b else 0
            table[b, :skip] = table[first[b], :skip]
            table[b, skip:np_b] = ids[at:at + np_b - skip]
            at += np_b - skip
            if first[b] != b and part[b]:  # an own copy of the page shared in part
                s, d = table[first[b], skip] * P, table[b, skip] * P
                self.codes[d:d + part[b]], self.scales[d:d + part[b]] = (self.codes[s:s + part[b]],
                                                                        self.scales[s:s + part[b]])
            j = np.arange(n[b])
            self.rows[b] = table[b, j // P].astype(np.int64) * P + j % P if n[b] else np.zeros(0, np.int64)
            seen[self.rows[b]] = True
        self.scales[~seen] = 0x7F
        self.table = table
        self.q = bf16(rng.standard_normal((B, H, D))) if q is None else q
        self.swa = F = None
        if n_swa:
            F = torch.from_numpy(rng.standard_normal((B, n_swa, D)).astype(np.float32)).to(torch.float8_e4m3fn)
            self.swa = F.view(torch.uint8).numpy()
        self.row_pos = self.lo = None
        if win:  # rows in ring order, some empty, some before the lowest visible position
            self.row_pos = rng.integers(-1, 300, (B, n_swa)).astype(np.int64)
            self.lo = rng.integers(-5, 250, B).astype(np.int64)
            self.lo[-1] = 1 << 40  # the last query sees no window row
        self.weight = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if extras else None
        self.q_pos = (1_000_003 + 37 * np.arange(B)).astype(np.int64) if extras else None
        self.sink = (2 * rng.standard_normal(H)).astype(np.float32) if sink else None

    def reference(self, n=None, of=None):
        outs, lses, bounds, lbs = [], [], [], []
        for b in range(self.B) if of is None else of:
            r = self.rows[b][:self.n[b] if n is None else n[b]]
            x = decode(self.codes[r], self.scales[r])
            if self.n_swa:
                vis = np.ones(self.n_swa, bool) if self.row_pos is None else self.row_pos[b] >= max(self.lo[b], 0)
                x = np.concatenate([x, F8[self.swa[b][vis]]])
            q = norm_rope_q(self.q[b].float().numpy(), self.weight, 1e-6, None if self.q_pos is None else self.q_pos[b],
                            10000.0)
            o, l, e, le = attention(x, q, SCALE, self.sink, self.weight is not None,
                                    None if self.q_pos is None else self.q_pos[b])
            outs.append(o)
            lses.append(l)
            bounds.append(e)
            lbs.append(le)
        return np.stack(outs), np.stack(lses), np.stack(bounds), np.stack(lbs)

    def device(self):
        t = {k: to_dev(getattr(self, k)) for k in ("codes", "scales", "table")}
        N = self.n_pages * self.P
        ix = torch.empty((N, 64), dtype=torch.uint8, device="cuda"), torch.empty((N, 4), dtype=torch.uint8, device="cuda")
        self.planes = csa2.Planes(t["codes"], t["scales"], *ix, self.P)
        self.pages = csa2.pages(t["table"], self.n_pages)
        self.dq = self.q.cuda()
        self.dn = to_dev(np.array(self.n, np.int32))
        self.dswa = to_dev(self.swa) if self.n_swa else None
        self.kw = dict(q_nr=csa2.norm_rope(to_dev(self.weight), 1e-6, True) if self.weight is not None else None,
                       q_pos=to_dev(self.q_pos) if self.q_pos is not None else None,
                       sink=to_dev(self.sink) if self.sink is not None else None,
                       win=csa2.window(to_dev(self.row_pos), to_dev(self.lo)) if self.row_pos is not None else None)
        return self

    def outputs(self, dtype):
        return (torch.full((self.B, H, D), 777.0, dtype=dtype, device="cuda"),
                torch.full((self.B, H), 777.0, dtype=torch.float32, device="cuda"))

    def paged(self, dtype=torch.float32, n_max=None, stream=None, ws=None):
        out, lse = self.outputs(dtype)
        n_max = max(self.n) if n_max is None else n_max
        ws = csa2.workspace(csa2.paged_attn_workspace_size(self.B, n_max, self.n_swa)) if ws is None else ws
        csa2.paged_attn_decode(self.planes, self.pages, self.B, self.dn, n_max, self.dswa, self.n_swa, self.dq, SCALE,
                               out, ws, lse_out=lse, stream=stream, **self.kw)
        return out, lse, ws

    def prefix(self, dtype=torch.float32, start=None, shared=None, shared_max=None, own_max=None, stream=None, keep=None,
               ws=None):
        out, lse = self.outputs(dtype)
        start = [a for a, _ in self.groups] + [self.groups[-1][1]] if start is None else start
        shared = self.shared if shared is None else shared
        if shared_max is None:
            shared_max = max(self.shared_max, *shared)
        own_max = max(self.n) if own_max is None else own_max
        G = len(shared)
        ws = csa2.workspace(csa2.prefix_attn_workspace_size(self.B, G, shared_max, own_max, self.n_swa)) if ws is None else ws
        self.keep = keep or (to_dev(np.array(start, np.int32)), to_dev(np.array(shared, np.int32)))
        csa2.prefix_attn_decode(self.planes, self.pages, self.B, self.dn, G, *self.keep, shared_max, own_max,
                                self.dswa, self.n_swa, self.dq, SCALE, out, ws, lse_out=lse, stream=stream, **self.kw)
        return out, lse, ws


def close(out, lse, ref, what=""):
    o, l, bound, lb = ref
    got = out.double().cpu().numpy()
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -22
    err = np.abs(got - o)
    lim = bound + half * (np.abs(o) + bound)
    assert np.isfinite(got).all(), what
    assert (err <= lim).all(), f"{what}: {(err / np.maximum(lim, 1e-300)).max():.2f} of the bound"
    g = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(g), np.isneginf(l)), what
    f = np.isfinite(l)
    assert (np.abs(g[f] - l[f]) <= lb[f]).all(), f"{what}: lse {np.abs(g[f] - l[f]).max():.2e}"


LENGTHS = [[0], [1], [63], [64], [65], [200, 0, 1, 127, 128, 129, 512], [1000, 3, 257]]


@pytest.mark.parametrize("P", [1, 7, 64, 100, 1024])
@pytest.mark.parametrize("n", LENGTHS)
def test_paged_lengths_and_page_sizes(n, P):
    b = Batch(17 * len(n) + P, n, P).device()
    out, lse, ws = b.paged()
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


@pytest.mark.parametrize("extras,sink", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("n_swa,win", [(128, False), (128, True), (5, True), (0, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_paged_window_extras_types(n_swa, win, extras, sink, dtype):
    b = Batch(5, [300, 0, 65, 17], 16, n_swa=n_swa, win=win, extras=extras, sink=sink).device()
    out, lse, ws = b.paged(dtype)
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


def test_paged_batch_beyond_the_gpu():
    rng = np.random.default_rng(1)
    n = [int(x) for x in rng.integers(0, 200, 333)]
    b = Batch(2, n, 16, n_swa=16).device()
    out, lse, ws = b.paged(torch.bfloat16)
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


def test_counts_beyond_the_bound_and_negative():
    b = Batch(3, [200, 90, 40], 16).device()
    b.dn = to_dev(np.array([200, 90, -7], np.int32))
    out, lse, ws = b.paged(n_max=120)
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference(n=[120, 90, 0]))


@pytest.mark.parametrize("page,detail", [(-3, -3), (10_000, 10_000)])
@pytest.mark.parametrize("prefix", [False, True])
def test_bad_page_is_reported_and_skipped(page, detail, prefix):
    b = Batch(4, [200, 90], 16, groups=[(0, 2)], shared=[0])
    b.device()
    t = b.table.copy()
    t[0, 2] = page
    b.pages = csa2.pages(to_dev(t), b.n_pages)
    b.rows[0] = np.concatenate([b.rows[0][:32], b.rows[0][48:]])
    b.n[0] = 184
    want = b.reference()
    b.n[0] = 200
    out, lse, ws = b.prefix() if prefix else b.paged()
    st, det = csa2.check(ws)
    assert st == 6 and det == detail
    close(out, lse, want)


@pytest.mark.parametrize("shared", [0, 90])
def test_bad_page_in_pairs(shared):
    # in the first query's own rows, or among the shared ones that all read from the widened image
    b = Batch(44, [200, 90, 90, 90, 90], 16, groups=[(0, 5)], shared=[shared])
    b.device()
    t = b.table.copy()
    t[0, 2] = -3
    b.pages = csa2.pages(to_dev(t), b.n_pages)
    for i in range(5 if shared else 1):
        b.rows[i] = np.concatenate([b.rows[i][:32], b.rows[i][48:]])
    want = b.reference(n=[10 ** 6] * 5)
    out, lse, ws = b.prefix()
    assert csa2.check(ws) == (6, -3)
    close(out, lse, want)


@pytest.mark.parametrize("others", [1, 5])
def test_long_cache_offsets_beyond_32_bits(others):
    # the pages sit behind 2^32 bytes of codes
    b = Batch(6, [150] + [70] * others, 64, [(0, 1 + others)], [64])
    N, P = b.n_pages, 64
    far = (1 << 32) // (256 * P) + 11
    b.device()
    codes = torch.zeros(((far + N) * P, 256), dtype=torch.uint8, device="cuda")
    scales = torch.full(((far + N) * P, 32), 0x7F, dtype=torch.uint8, device="cuda")
    codes[far * P:], scales[far * P:] = to_dev(b.codes), to_dev(b.scales)
    b.planes = csa2.Planes(codes, scales, codes, scales, P)  # the indexer planes are not read
    t = b.table.copy()
    t[t < N] += far
    b.pages = csa2.pages(to_dev(t), far + N)
    want = b.reference()
    for out, lse, ws in (b.paged(), b.prefix()):
        assert csa2.check(ws)[0] == 0
        close(out, lse, want)


GROUPS = [
    # n, groups, shared
    ([40, 40], [(0, 2)], [40]),                                   # nothing of their own
    ([1, 1, 1], [(0, 3)], [1]),
    ([300, 310, 300, 305, 299], [(0, 5)], [299]),                 # odd group, odd length
    ([128, 140], [(0, 2)], [128]),
    ([129, 140], [(0, 2)], [129]),
    ([500, 500, 90, 700, 650, 33], [(0, 2), (2, 3), (3, 5), (5, 6)], [450, 80, 640, 33]),
    ([260, 100, 260, 0, 77], [(0, 5)], [256]),                    # some see only a part of the prefix
    ([260, 261, 0, 0], [(0, 2)], [256]),                          # padded queries outside every group
    ([50, 260, 261, 20], [(1, 3)], [100]),
    ([400, 400], [(0, 2)], [0]),                                  # a group that shares nothing
    ([1500, 1501, 1502, 1503, 1504, 1505, 1506], [(0, 7)], [1490]),
]


@pytest.mark.parametrize("times", [1, 5])
@pytest.mark.parametrize("P", [16, 100])
@pytest.mark.parametrize("n,groups,shared", GROUPS)
def test_prefix_groups(n, groups, shared, P, times):
    b = Batch(len(n) * 7 + P, *repeated(n, groups, shared, times)[:1], P, *repeated(n, groups, shared, times)[1:]).device()
    out, lse, ws = b.prefix()
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


@pytest.mark.parametrize("n,groups,shared,own_max", [
    ([100, 300, 310, 40], [(0, 4)], [280], 30),   # the first query sees a part only: others' rows hold the rest
    ([50, 300], [(0, 2)], [280], 20),
    ([0, 0, 300, 290, 0], [(0, 5)], [280], 20),
    ([100, 200, 150], [(0, 3)], [280], 0),        # none has them all
    ([0, 0, 0], [(0, 3)], [280], 0),
])
@pytest.mark.parametrize("times", [1, 5])
def test_prefix_longer_than_the_first_query(n, groups, shared, own_max, times):
    n, groups, shared = repeated(n, groups, shared, times)
    b = Batch(40, n, 16, groups, shared, n_swa=5).device()
    out, lse, ws = b.prefix(own_max=own_max, shared_max=max(b.shared_max, 280) if times > 1 else min(280, 16 * b.max_pages))
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


@pytest.mark.parametrize("times", [1, 5])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_one_head_of_a_query_not_finite(value, times):
    b = Batch(41, [300, 310, 320] * times, 16, [(0, 3 * times)], [256], n_swa=16)
    want = b.reference()
    b.q[1, 7, 3] = value
    b.device()
    for out, lse, ws in (b.prefix(), b.paged()):
        assert csa2.check(ws)[0] == 0
        assert torch.isnan(out[1, 7]).all()
        out[1, 7] = torch.from_numpy(want[0][1, 7]).float().cuda()
        lse[1, 7] = float(want[1][1, 7])
        close(out, lse, want)


@pytest.mark.parametrize("B", [3, 20])
def test_without_lse_the_same_output(B):
    b = Batch(42, [300 + i for i in range(B)], 16, [(0, B)], [290], n_swa=16, extras=True, sink=True).device()
    ws = csa2.workspace(max(csa2.prefix_attn_workspace_size(B, 1, b.shared_max, 300, 16), csa2.paged_attn_workspace_size(B, 400, 16)))
    keep = to_dev(np.array([0, B], np.int32)), to_dev(np.array([290], np.int32))
    out = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda")
    one = b.prefix(torch.bfloat16)
    csa2.prefix_attn_decode(b.planes, b.pages, B, b.dn, 1, *keep, b.shared_max, 300, b.dswa, 16, b.dq, SCALE, out, ws, **b.kw)
    assert csa2.check(ws)[0] == 0 and torch.equal(out, one[0])
    one = b.paged(torch.bfloat16)
    csa2.paged_attn_decode(b.planes, b.pages, B, b.dn, 299 + B, b.dswa, 16, b.dq, SCALE, out, ws, **b.kw)
    assert csa2.check(ws)[0] == 0 and torch.equal(out, one[0])


@pytest.mark.parametrize("extras,sink", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("n_swa,win", [(128, False), (128, True), (7, True)])
@pytest.mark.parametrize("dtype,times", [(torch.float32, 1), (torch.bfloat16, 1), (torch.bfloat16, 5)])
def test_prefix_window_extras_types(n_swa, win, extras, sink, dtype, times):
    n, groups, shared = repeated([300, 290, 289, 0, 65, 17], [(0, 3), (3, 5)], [280, 60], times)
    b = Batch(9, n, 16, groups, shared, n_swa=n_swa, win=win, extras=extras, sink=sink).device()
    out, lse, ws = b.prefix(dtype)
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


@pytest.mark.parametrize("times", [1, 3])
def test_prefix_large_logits_move_the_reference(times):
    # later entries with ever larger logits: the running maximum moves again and again
    b = Batch(12, [700, 690, 710] * times, 16, [(0, 3 * times)], [650])
    b.q = bf16(b.q.float().numpy() * 6.0)
    r = b.rows[0]
    for j in range(0, 650, 50):  # scale factors 2^0 .. 2^3 growing along the sequence
        rows = np.unique(np.concatenate([x[j:j + 50] for x in b.rows]))
        b.scales[rows] = np.minimum(b.scales[rows] + 8 * (j // 160), 0x70)
    b.device()
    for out, lse, ws in (b.prefix(), b.paged()):
        assert csa2.check(ws)[0] == 0
        close(out, lse, b.reference())


@pytest.mark.parametrize("most", [4, 12])
def test_prefix_many_small_groups_and_one_large(most):
    rng = np.random.default_rng(8)
    n, groups, shared, at = [], [], [], 0
    for g in range(60):
        size, sh = int(rng.integers(1, most + 1)), int(rng.integers(0, 200))
        n += [sh + int(rng.integers(0, 90)) for _ in range(size)]
        groups.append((at, at + size))
        shared.append(sh)
        at += size
    n += [1000 + int(rng.integers(0, 40)) for _ in range(31)]
    groups.append((at, at + 31))
    shared.append(1000)
    b = Batch(13, n, 16, groups, shared, n_swa=32).device()
    out, lse, ws = b.prefix(torch.bfloat16)
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


@pytest.mark.parametrize("times", [1, 440])  # 1,320 queries: pairs also with the bound of 100
def test_prefix_bounds_of_the_host(times):
    q = torch.randn((64, H, D), generator=torch.Generator().manual_seed(14)).to(torch.bfloat16)
    B = 3 * times
    b = Batch(14, [300, 310, 320] * times, 16, [(0, B)], [256], q=q.repeat(-(-B // 64), 1, 1)[:B]).device()
    of = np.arange(B) if times == 1 else np.arange(0, B, 41)
    at = torch.from_numpy(of).cuda()
    # n_shared above its bound: the rest is read as each query's own
    out, lse, ws = b.prefix(shared_max=100, own_max=220)
    assert csa2.check(ws)[0] == 0
    close(out[at], lse[at], b.reference(of=of))
    # own entries above theirs: left out and reported
    out, lse, ws = b.prefix(shared_max=256, own_max=50)
    st, det = csa2.check(ws)
    assert st == 6 and det in (310, 320)
    close(out[at], lse[at], b.reference(n=[300, 306, 306] * times, of=of))
    # a negative count of shared entries is none
    out, lse, ws = b.prefix(shared=[-4], shared_max=0 if times == 1 else 100)
    assert csa2.check(ws)[0] == 0
    close(out[at], lse[at], b.reference(of=of))


@pytest.mark.parametrize("start,shared", [([0, -1, 3], [256, 256]), ([0, 9, 3], [256, 256]), ([2, 0, 3], [256, 256])])
@pytest.mark.parametrize("times", [1, 4])  # twelve queries in two groups run in pairs
def test_prefix_bad_groups_are_empty_and_reported(start, shared, times):
    b = Batch(15, [300, 310, 320] * times, 16, [(0, 3 * times)], [256]).device()
    start = [x if x < 3 else (x if x == 9 and times == 1 else 99 if x == 9 else 3 * times) for x in start]
    out, lse, ws = b.prefix(start=start, shared=shared)
    assert csa2.check(ws)[0] == 6
    close(out, lse, b.reference())


def test_no_lse_and_untouched_rows():
    b = Batch(16, [100, 90], 16, [(0, 2)], [80]).device()
    out = torch.full((4, H, D), 777.0, dtype=torch.bfloat16, device="cuda")
    ws = csa2.workspace(csa2.prefix_attn_workspace_size(2, 1, 80, 20, 0))
    keep = to_dev(np.array([0, 2], np.int32)), to_dev(np.array([80], np.int32))
    csa2.prefix_attn_decode(b.planes, b.pages, 2, b.dn, 1, *keep, 80, 20, None, 0, b.dq, SCALE, out, ws)
    ref = b.reference()
    got = out.double().cpu().numpy()
    assert (got[2:] == 776.0).all()  # 777 in bf16: eight bits, steps of 4
    assert (np.abs(got[:2] - ref[0]) <= ref[2] + 2.0 ** -8 * (np.abs(ref[0]) + ref[2])).all()


def test_graph_replay_with_new_lengths_and_two_streams():
    b = Batch(18, [300, 310, 320, 64, 50, 10], 16, [(0, 3)], [256], n_swa=16).device()
    st, st2 = torch.cuda.Stream(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    st2.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b.prefix(stream=st, own_max=70)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out, lse, ws = b.prefix(stream=st, own_max=70, keep=b.keep)  # no copies while capturing
    with torch.cuda.stream(st2):
        out2, lse2, ws2 = b.paged()
    st2.synchronize()
    close(out2, lse2, b.reference())
    b.dn.copy_(torch.tensor([256, 0, 311, 1, 0, 7], dtype=torch.int32))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(3):
            g.replay()
    st.synchronize()
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference(n=[256, 0, 311, 1, 0, 7]))


@pytest.mark.parametrize("more", [0, 4])
def test_same_results_call_after_call(more):
    b = Batch(19, [900, 901, 902] + [890] * more, 16, [(0, 3 + more)], [880], n_swa=128).device()
    one = b.prefix(torch.bfloat16)
    assert csa2.check(one[2])[0] == 0
    for _ in range(5):
        two = b.prefix(torch.bfloat16)
        assert csa2.check(two[2])[0] == 0
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


@pytest.mark.parametrize("prefix,B", [(False, 2), (False, 20), (True, 2), (True, 5), (True, 20)])
def test_logsumexp_of_one_rounded_row(prefix, B):
    """Every head's query is normalised and rotated, which its f16 form rounds; each query's one row has the
    signs of what head 0's rounding takes, so that it all adds up: some 2^-9.  The logsumexp is corrected for
    it: left are the fp32 sums' 2^-16 of scale sum |q x|, with e = 2^-11 of that at most e^2 / 2 (half the
    square of half the width 2 e) and, of the correction itself, e (2^-11 for its f16 terms + 2^-9 for o)."""
    b = Batch(21, [1] * B, 16, [(0, B)], [0], extras=True)
    lost = []
    for i in range(B):
        q = norm_rope_q(b.q[i].float().numpy(), b.weight, 1e-6, b.q_pos[i], 10000.0)[0]
        r = q - q.astype(np.float16).astype(np.float64)
        code = np.where(r < 0, 12, 4).astype(np.uint8)  # -2, 2
        b.codes[b.rows[i][0]], b.scales[b.rows[i][0]] = code[0::2] | code[1::2] << 4, 0x38
        lost.append(SCALE * 2 * np.abs(r).sum())
    b.device()
    out, lse, ws = b.prefix() if prefix else b.paged()
    assert csa2.check(ws)[0] == 0
    ref = b.reference()
    close(out, lse, ref)
    for i in range(B):
        q = norm_rope_q(b.q[i].float().numpy(), b.weight, 1e-6, b.q_pos[i], 10000.0)
        x = decode(b.codes[b.rows[i]], b.scales[b.rows[i]])
        z = SCALE * (np.abs(q) @ np.abs(x).T)[:, 0]
        e = z * 2.0 ** -11
        tol = z * 2.0 ** -16 + e * e / 2 + e * (2.0 ** -11 + 2.0 ** -9) + 2.0 ** -22 * np.abs(ref[1][i])
        assert lost[i] > 4 * tol[0]
        assert (np.abs(lse[i].double().cpu().numpy() - ref[1][i]) <= tol).all()


@pytest.mark.parametrize("n_swa", [0, 128])
@pytest.mark.parametrize("pairs", [False, True])
def test_nan_reaches_only_the_queries_that_see_it(n_swa, pairs):
    n = [300, 100, 300, 150, 90, 700, 95, 99] + [88] * (2 if pairs else 0)
    b = Batch(22, n, 16, [(0, 4), (4, len(n))], [280, 80], n_swa=n_swa)
    bad = {0, 2, 5}
    b.scales[b.rows[0][200], 3] = 0x7F   # shared, seen by 0 and 2
    b.scales[b.rows[5][600], 31] = 0xFF  # the own of 5
    b.scales[b.rows[5][85], 0] = 0x7F    # and among the rows next to those of 4
    if n_swa:
        b.swa[7, 100, 511] = 0xFF
        bad.add(7)
    b.device()
    good = [i for i in range(len(n)) if i not in bad]
    want = b.reference(of=good)
    for out, lse, ws in (b.prefix(), b.paged()):
        assert csa2.check(ws)[0] == 0
        close(out[good], lse[good], want)
        assert torch.isnan(out[sorted(bad)]).all() and torch.isnan(lse[sorted(bad)]).all()


@pytest.mark.parametrize("more", [0, 4])
def test_padded_queries_may_hold_nan(more):
    b = Batch(23, [0, 70, 0] + [66] * more, 16, [(1, 3 + more)], [64], extras=True, sink=True)
    q = b.q.clone()
    b.q[0], b.q[2] = 0, 0
    want = b.reference()
    b.q = q
    b.q[0], b.q[2, :, 5] = float("nan"), float("inf")
    b.device()
    for out, lse, ws in (b.prefix(), b.paged()):
        assert csa2.check(ws)[0] == 0
        close(out, lse, want)


def test_sinks_of_minus_infinity_and_no_rows():
    b = Batch(24, [0, 40], 16, [(0, 2)], [0], sink=True)
    b.sink[::2] = -np.inf
    b.device()
    with np.errstate(divide="ignore"):
        want = b.reference(of=[1])
    for out, lse, ws in (b.prefix(), b.paged()):
        assert csa2.check(ws)[0] == 0
        close(out[1:], lse[1:], want)
        l0 = lse[0].cpu().numpy()
        assert (out[0] == 0).all() and np.isneginf(l0[::2]).all()
        assert np.abs(l0[1::2] - b.sink[1::2]).max() <= 2.0 ** -20


@pytest.mark.parametrize("P,n_pages", [(20000, 5), (70001, 3), (1 << 22, 1)])
def test_large_pages(P, n_pages):
    b = Batch(25, [300, 260], 64, [(0, 2)], [256])
    want = b.reference()
    N = n_pages * P
    b.device()
    codes = torch.zeros((N, 256), dtype=torch.uint8, device="cuda")
    scales = torch.full((N, 32), 0x7F, dtype=torch.uint8, device="cuda")
    # one sequence after the other: query 1 has its own page where there is one, else sees query 0's entries
    t = [n_pages - 1, max(n_pages - 2, 0)]
    rows = [t[i] * P + np.arange(b.n[i]) for i in range(2)]
    if n_pages == 1:
        b.rows[1] = b.rows[0][:260]
        want = b.reference()
    for i in range(2):
        at = torch.from_numpy(rows[i]).cuda()
        codes[at], scales[at] = to_dev(b.codes[b.rows[i]]), to_dev(b.scales[b.rows[i]])
    b.planes = csa2.Planes(codes, scales, codes, scales, P)
    b.pages = csa2.pages(to_dev(np.array(t, np.int32)[:, None]), n_pages)
    b.max_pages = 1
    for out, lse, ws in (b.prefix(), b.paged()):
        assert csa2.check(ws)[0] == 0
        close(out, lse, want)


def test_one_long_query_among_many():
    n = [9000] + [3] * 19
    b = Batch(26, n, 16, [(0, 20)], [2], n_swa=4).device()
    want = b.reference()
    for out, lse, ws in (b.prefix(), b.paged()):
        assert csa2.check(ws)[0] == 0
        close(out, lse, want)


@pytest.mark.parametrize("prefix,B", [(False, 9000), (True, 9000), (True, 21000)])
def test_batches_beyond_the_plans_shared_memory(prefix, B):
    # each query a group, or five of them (4,200 groups): most of them empty, the last ones not
    rng = np.random.default_rng(27)
    n = np.zeros(B, int)
    live = np.concatenate([rng.choice(B - 40, 60, replace=False), np.arange(B - 5, B)])
    n[live] = rng.integers(1, 300, live.size)
    q = torch.randn((64, H, D), generator=torch.Generator().manual_seed(27)).to(torch.bfloat16)
    size = 5 if B > 9000 else 1
    if size > 1:  # whole groups of the same length
        n = np.repeat(n[::size], size)
        live = np.flatnonzero(n)
    b = Batch(27, [int(x) for x in n], 16, [(i, i + size) for i in range(0, B, size)], [int(x) // 2 for x in n[::size]],
              q=q.repeat(-(-B // 64), 1, 1)[:B]).device()
    out, lse, ws = b.prefix(torch.bfloat16) if prefix else b.paged(torch.bfloat16)
    assert csa2.check(ws)[0] == 0
    at = torch.from_numpy(live).cuda()
    close(out[at], lse[at], b.reference(of=live))
    dead = torch.from_numpy(np.flatnonzero(n == 0)).cuda()
    assert (lse[dead] == -np.inf).all() and not out[dead].any()


@pytest.mark.parametrize("most", [5, 14])
def test_groups_beyond_one_strip_of_the_plan(most):
    # 700 groups, of one to four or to thirteen queries, over the pages of one long prompt
    rng = np.random.default_rng(28)
    size = rng.integers(1, most, 700)
    start = np.concatenate([[0], np.cumsum(size)])
    B = int(start[-1])
    group = np.repeat(np.arange(700), size)
    shared = rng.integers(0, 180, 700)
    n = shared[group] + rng.integers(0, 20, B)
    one = Batch(28, [200], 16)
    q = torch.randn((64, H, D), generator=torch.Generator().manual_seed(28)).to(torch.bfloat16)
    one.device()
    one.B, one.n, one.dn, one.q = B, [int(x) for x in n], to_dev(n.astype(np.int32)), q.repeat(-(-B // 64), 1, 1)[:B]
    one.dq, one.rows = one.q.cuda(), [one.rows[0][:x] for x in n]
    one.groups, one.shared = [(int(start[g]), int(start[g + 1])) for g in range(700)], [int(x) for x in shared]
    one.pages = csa2.pages(to_dev(np.repeat(one.table, B, 0)), one.n_pages)
    out, lse, ws = one.prefix(torch.bfloat16, own_max=20)
    assert csa2.check(ws)[0] == 0
    of = np.concatenate([np.arange(30), rng.choice(B, 100), np.arange(B - 30, B)])
    at = torch.from_numpy(of).cuda()
    close(out[at], lse[at], one.reference(of=of))


def test_more_shared_entries_than_the_workspace_widens():
    # 18 groups of five queries on 65,536 entries each, the same pages: beyond 2^20 entries, the last
    # groups' entries are widened where they are read
    G, ns = 18, 65536
    one = Batch(29, [ns], 64)
    q = torch.randn((5 * G, H, D), generator=torch.Generator().manual_seed(29)).to(torch.bfloat16)
    one.device()
    B = one.B = 5 * G
    one.n, one.dn, one.q, one.dq = [ns] * B, to_dev(np.full(B, ns, np.int32)), q, q.cuda()
    one.groups, one.shared = [(5 * g, 5 * g + 5) for g in range(G)], [ns] * G
    one.pages = csa2.pages(to_dev(np.repeat(one.table, B, 0)), one.n_pages)
    x = decode(one.codes[one.rows[0]], one.scales[one.rows[0]])
    out, lse, ws = one.prefix(own_max=0)
    assert csa2.check(ws)[0] == 0
    of = [0, 24, 81, 89]
    close(out[of], lse[of], tuple(np.stack(z) for z in zip(*(attention(x, q[i].double().numpy(), SCALE) for i in of))))


def test_two_graphs_share_a_workspace():
    b = Batch(30, [300, 310, 320, 64, 0], 16, [(0, 3)], [256], n_swa=16, extras=True, sink=True).device()
    size = max(csa2.prefix_attn_workspace_size(5, 1, b.shared_max, 70, 16), csa2.paged_attn_workspace_size(5, 320, 16))
    ws = csa2.workspace(size)
    b.prefix(own_max=70, ws=ws)
    b.paged(ws=ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    with torch.cuda.stream(st):
        for i, g in enumerate(graphs):
            with torch.cuda.graph(g, stream=st):
                outs.append(b.paged(ws=ws) if i else b.prefix(own_max=70, ws=ws, keep=b.keep))
        for i in (0, 1, 1, 0, 1, 0):
            graphs[i].replay()
    st.synchronize()
    want = b.reference()
    for out, lse, _ in outs:
        close(out, lse, want)
    assert csa2.check(ws)[0] == 0


def test_calls_at_once_on_streams_of_their_own():
    b = Batch(31, [900, 901, 902, 64] * 4, 16, [(0, 3), (3, 4), (4, 7)], [880, 10, 400], n_swa=16).device()
    want = b.reference()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    b.prefix()
    torch.cuda.synchronize()
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(b.prefix(keep=b.keep) if i % 2 else b.paged())
    torch.cuda.synchronize()
    for out, lse, ws in got:
        assert csa2.check(ws)[0] == 0
        close(out, lse, want)


def test_whole_run_tables_append_window_attention(oracle_mod):
    """Two decode steps of four requests on a shared prompt: tables and maps on the GPU, the new entries
    appended through them, the window, then attention; the reference reads the planes' own bytes."""
    rng = np.random.default_rng(20)
    B, P, d, m, n_pages, max_pages = 4, 16, 128, 2, 40, 8
    prompt = 37  # shared: two whole pages and five entries of a third
    planes = csa2.Planes.empty(n_pages, P)
    lat = to_dev(rng.standard_normal((n_pages * P, 512)).astype(np.float32))
    ki = to_dev(rng.standard_normal((n_pages * P, 128)).astype(np.float32))
    csa2.quantize_entries(planes, lat, ki, n_pages * P)
    table = np.full((B, max_pages), -1, np.int32)
    table[:, :2] = [7, 3]
    table[:, 2] = [11, 12, 13, 14]
    for b in range(1, B):  # own copies of the page shared in part
        for t in (planes.kv_codes, planes.kv_scales):
            t[(11 + b) * P:(11 + b) * P + 5] = t[11 * P:11 * P + 5]
    table_d = to_dev(table)
    free = to_dev(np.array([p for p in range(n_pages) if p not in (7, 3, 11, 12, 13, 14)] + [-1] * 6, np.int32))
    n_free, have = to_dev(np.array([34], np.int32)), to_dev(np.full(B, prompt, np.int32))
    kept = to_dev(np.full(B, 2, np.int32))
    e = lambda n, t: torch.empty(n, dtype=t, device="cuda")
    Wkv, Wz, Wik = (to_dev(rng.standard_normal(s).astype(np.float32) * d ** -0.5).to(torch.bfloat16)
                    for s in ((d, 512), (d, 512), (512, 128)))
    ring = torch.zeros((B, 128, 512), dtype=torch.uint8, device="cuda")
    ring_pos = torch.full((B, 128), -1, dtype=torch.int64, device="cuda")
    lo = torch.zeros(B, dtype=torch.int64, device="cuda")
    counts = [prompt] * B
    for add in ([1, 12, 0, 30], [3, -4, 1, 1]):
        rows = sum(max(a, 0) for a in add)
        query, slot, entry, pos = e(rows, torch.int32), e(rows, torch.int32), e(rows, torch.int64), e(rows, torch.int64)
        ws = csa2.workspace(csa2.page_tables_workspace_size(B))
        csa2.page_tables(B, have, to_dev(np.array(add, np.int32)), P, table_d, max_pages, n_pages, free, n_free, n_free,
                         have, ws, n_rows=rows, query=query, slot=slot, entry=entry, pos=pos, m=m, n_kept=kept)
        Hd = to_dev(rng.standard_normal((rows, m, d)).astype(np.float32)).to(torch.bfloat16)
        wsa = csa2.workspace(csa2.cache_append_workspace_size(rows, d, m))
        csa2.cache_append(Hd, rows, d, Wkv, Wz, Wik, m, planes, n_pages, slot, entry, wsa)
        csa2.swa_append(to_dev(rng.standard_normal((rows, 512)).astype(np.float32)), rows, pos, B, ring, 128,
                        query=query, ring_pos=ring_pos)
        q = bf16(rng.standard_normal((B, H, D)))
        out, lse = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda"), e((B, H), torch.float32)
        wsp = csa2.workspace(csa2.prefix_attn_workspace_size(B, 1, prompt, 64, 128))
        csa2.prefix_attn_decode(planes, csa2.pages(table_d, n_pages), B, have, 1, to_dev(np.array([0, B], np.int32)),
                                to_dev(np.array([prompt], np.int32)), prompt, 64, ring, 128, q.cuda(), SCALE, out, wsp,
                                lse_out=lse, win=csa2.window(ring_pos, lo))
        for w in (ws, wsa, wsp):
            assert csa2.check(w)[0] == 0
        counts = [c + a for c, a in zip(counts, add)]
        assert have.cpu().tolist() == counts
        t, codes, scales = table_d.cpu().numpy(), planes.kv_codes.cpu().numpy(), planes.kv_scales.cpu().numpy()
        swa, rp = ring.cpu().numpy(), ring_pos.cpu().numpy()
        ref = []
        for b in range(B):
            j = np.arange(counts[b])
            r = t[b, j // P].astype(np.int64) * P + j % P
            assert len(set(r)) == counts[b]
            x = np.concatenate([decode(codes[r], scales[r]), F8[swa[b][rp[b] >= 0]]])
            ref.append(attention(x, q[b].double().numpy(), SCALE))
        close(out, lse, tuple(np.stack(z) for z in zip(*ref)))


@pytest.mark.parametrize("pairs", [False, True])
def test_more_entries_than_either_bound(pairs):
    # shared and own entries together reach beyond 65,536, in pages of an odd size
    n = [100_003, 65_537] + ([65_500] * 3 if pairs else [])
    b = Batch(43, n, 97, [(0, len(n))], [65_500]).device()
    out, lse, ws = b.prefix(own_max=34_600)
    assert csa2.check(ws)[0] == 0
    close(out[:3], lse[:3], b.reference(of=range(min(3, len(n)))))


@pytest.mark.parametrize("B,kernel", [(4, "k_paged_attn"), (5, "k_prefix_attn")])
def test_which_form_runs(B, kernel):
    # the tests of pairs run pairs
    b = Batch(45, [300] * B, 16, [(0, B)], [290]).device()
    csa2.timing_enable(True)
    try:
        b.prefix()
        torch.cuda.synchronize()
        assert {"k_paged_attn", "k_prefix_attn"} & set(csa2.kernel_times()) == {kernel}
    finally:
        csa2.timing_enable(False)
