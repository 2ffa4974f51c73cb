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


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


class Batch:
    """A paged cache on both sides: B sequences of n[b] entries in pages of P, groups of queries that
    share their first entries.  Every entry that no query may see has a NaN scale."""

    def __init__(self, seed, n, P, groups=(), shared=(), n_swa=0, win=False, extras=False, sink=False, spare=3):
        rng = np.random.default_rng(seed)
        self.B, self.P, self.n, self.n_swa, self.groups, self.shared = len(n), P, list(n), n_swa, groups, list(shared)
        B = self.B
        self.max_pages = max(1, max(-(-x // P) for x in n))
        first, whole, part = list(range(B)), [0] * B, [0] * B
        for g, (a, z) in enumerate(groups):
            for b in range(a, z):
                first[b] = a
                agree = min(shared[g], n[a], n[b])
                whole[b], part[b] = agree // P, agree % P
        count = sum(-(-n[b] // P) - (whole[b] if first[b] != b else 0) for b in range(B)) + spare
        ids = rng.permutation(count).astype(np.int32)
        self.n_pages = count
        self.codes, self.scales = random_entries(rng, count * P)
        seen = np.zeros(count * P, bool)
        # garbage behind the last page of a sequence is not read
        table = np.full((B, self.max_pages), 0x7fffffff, np.int32)
        at = 0
        self.rows = []
        for b in range(B):
            np_b, skip = -(-n[b] // P), whole[b] if first[b] != b else 0
            table[b, :skip] = table[first[b], :skip]
            table[b, skip:np_b] = ids[at:at + np_b - skip]
            at += np_b - skip
            if first[b] != b and part[b]:  # an own copy of the page shared in part
                s, d = table[first[b], skip] * P, table[b, skip] * P
                self.codes[d:d + part[b]], self.scales[d:d + part[b]] = (self.codes[s:s + part[b]],
                                                                        self.scales[s:s + part[b]])
            j = np.arange(n[b])
            self.rows.append(table[b, j // P].astype(np.int64) * P + j % P if n[b] else np.zeros(0, np.int64))
            seen[self.rows[-1]] = True
        self.scales[~seen] = 0x7F
        self.table = table
        self.q = bf16(rng.standard_normal((B, H, D)))
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

    def reference(self, n=None, shared=None):
        outs, lses, bounds, lbs = [], [], [], []
        for b in range(self.B):
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

    def prefix(self, dtype=torch.float32, start=None, shared=None, shared_max=None, own_max=None, stream=None, keep=None):
        out, lse = self.outputs(dtype)
        start = [a for a, _ in self.groups] + [self.groups[-1][1]] if start is None else start
        shared = self.shared if shared is None else shared
        shared_max = max(max(self.shared), 0) if shared_max is None else shared_max
        own_max = max(self.n) if own_max is None else own_max
        G = len(shared)
        ws = csa2.workspace(csa2.prefix_attn_workspace_size(self.B, G, shared_max, own_max, self.n_swa))
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


def test_long_cache_offsets_beyond_32_bits():
    # the pages sit behind 2^32 bytes of codes
    b = Batch(6, [150, 70], 64, groups=[(0, 2)], shared=[64])
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


@pytest.mark.parametrize("P", [16, 100])
@pytest.mark.parametrize("n,groups,shared", GROUPS)
def test_prefix_groups(n, groups, shared, P):
    b = Batch(len(n) * 7 + P, n, P, groups, shared).device()
    out, lse, ws = b.prefix()
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


@pytest.mark.parametrize("extras,sink", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("n_swa,win", [(128, False), (128, True), (7, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefix_window_extras_types(n_swa, win, extras, sink, dtype):
    b = Batch(9, [300, 290, 289, 0, 65, 17], 16, [(0, 3), (3, 5)], [280, 60], n_swa=n_swa, win=win, extras=extras,
              sink=sink).device()
    out, lse, ws = b.prefix(dtype)
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


def test_prefix_large_logits_move_the_reference():
    # later entries with ever larger logits: the running maximum moves again and again
    b = Batch(12, [700, 690, 710], 16, [(0, 3)], [650])
    b.q = bf16(b.q.float().numpy() * 6.0)
    r = b.rows[0]
    for j in range(0, 650, 50):  # scale factors 2^0 .. 2^3 growing along the sequence
        rows = np.unique(np.concatenate([x[j:j + 50] for x in b.rows]))
        b.scales[rows] = np.minimum(b.scales[rows] + 8 * (j // 160), 0x70)
    b.device()
    for out, lse, ws in (b.prefix(), b.paged()):
        assert csa2.check(ws)[0] == 0
        close(out, lse, b.reference())


def test_prefix_many_small_groups_and_one_large():
    rng = np.random.default_rng(8)
    n, groups, shared, at = [], [], [], 0
    for g in range(60):
        size, sh = int(rng.integers(1, 5)), int(rng.integers(0, 200))
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


def test_prefix_bounds_of_the_host():
    b = Batch(14, [300, 310, 320], 16, [(0, 3)], [256]).device()
    # n_shared above its bound: the rest is read as each query's own
    out, lse, ws = b.prefix(shared_max=100, own_max=220)
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())
    # own entries above theirs: left out and reported
    out, lse, ws = b.prefix(shared_max=256, own_max=50)
    st, det = csa2.check(ws)
    assert st == 6 and det in (310, 320)
    close(out, lse, b.reference(n=[300, 306, 306]))
    # a negative count of shared entries is none
    out, lse, ws = b.prefix(shared=[-4], shared_max=0)
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference())


@pytest.mark.parametrize("start,shared", [([0, -1, 3], [256, 256]), ([0, 9, 3], [256, 256]), ([2, 0, 3], [256, 256])])
def test_prefix_bad_groups_are_empty_and_reported(start, shared):
    b = Batch(15, [300, 310, 320], 16, [(0, 3)], [256]).device()
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
    b = Batch(18, [300, 310, 320, 64], 16, [(0, 3)], [256], n_swa=16).device()
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
    b.dn.copy_(torch.tensor([256, 0, 311, 1], dtype=torch.int32))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(3):
            g.replay()
    st.synchronize()
    assert csa2.check(ws)[0] == 0
    close(out, lse, b.reference(n=[256, 0, 311, 1]))


def test_same_results_call_after_call():
    b = Batch(19, [900, 901, 902], 16, [(0, 3)], [880], n_swa=128).device()
    one = b.prefix(torch.bfloat16)
    assert csa2.check(one[2])[0] == 0
    for _ in range(5):
        two = b.prefix(torch.bfloat16)
        assert csa2.check(two[2])[0] == 0
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


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
