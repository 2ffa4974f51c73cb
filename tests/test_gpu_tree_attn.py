"""csa2_tree_attn_decode against attention in float64 over the rows that each drafted token sees, within the bound that
the kernels' roundings allow (paged_common.attention), at tree shapes, contexts, page sizes and windows where it can go
wrong; what is found on the device; graphs and streams."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from paged_common import D, F8, H, attention, decode, random_entries
from rotary_common import rotate

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5
YARN = ("yarn", 16.0, 65536, 32.0, 1.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def chain(T):
    return list(range(-1, T - 1))


def star(T):
    return [-1] * T


def binary(T):
    return [(t - 1) // 2 if t else -1 for t in range(T)]


def random_tree(rng, T):
    return [-1 if t == 0 or rng.random() < 0.15 else int(rng.integers(0, t)) for t in range(T)]


def path_to(parents, t):
    out = []
    while t >= 0:
        out.insert(0, t)
        t = parents[t]
    return out


class Forest:
    """Requests of n[g] entries in pages of P with draft trees, on both sides.  Entries that no query may see have a NaN
    scale, ring rows too."""

    def __init__(self, seed, n, trees, P=16, n_swa=128, entries=True, extras=False, sink=False, pad=0, pairs=False, spare=3):
        rng = np.random.default_rng(seed)
        R = self.R = len(n)
        self.n, self.trees, self.P, self.n_swa, self.entries, self.pad = list(n), trees, P, n_swa, entries, pad
        T = [len(t) for t in trees]
        self.start = np.concatenate([[0], np.cumsum(T)]).astype(np.int32)
        self.B = int(self.start[-1]) + pad
        total = [h + t * entries for h, t in zip(n, T)]
        self.n_max = max(n)
        if pairs:  # queries run in pairs where there are five to a request and n_max makes for enough work
            self.n_max = max(self.n_max, -(-(R << 21) // self.B ** 2))
            assert self.B >= 5 * R and self.n_max <= 65536
        self.most = max(1, max(T))
        self.max_pages = -(-(self.n_max + csa2.MAX_TREE) // P)
        count = sum(-(-t // P) for t in total) + spare
        self.n_pages = count
        ids = rng.permutation(count).astype(np.int32)
        self.table = np.full((R, self.max_pages), 0x7fffffff, np.int32)
        self.codes, self.scales = random_entries(rng, count * P)
        there = np.zeros(count * P, bool)
        at, self.rows = 0, []
        for g in range(R):
            k = -(-total[g] // P)
            self.table[g, :k] = ids[at:at + k]
            at += k
            e = np.arange(total[g])
            self.rows.append(self.table[g, e // P].astype(np.int64) * P + e % P if total[g] else np.zeros(0, np.int64))
            there[self.rows[g]] = True
        self.scales[~there] = 0x7F
        self.q = torch.from_numpy(rng.standard_normal((self.B, H, D)).astype(np.float32)).to(torch.bfloat16)
        self.parent = np.array([p for t in trees for p in t] + [-9] * pad, np.int32)
        self.paths = [path_to(t, i) for t in trees for i in range(len(t))]
        self.pos0 = (rng.integers(0, 2 * max(n_swa, 1), R) if not extras else rng.integers(1 << 19, 1 << 20, R)).astype(np.int64)
        group = np.repeat(np.arange(R), T)
        self.group = group
        self.q_pos = np.concatenate([[self.pos0[g] + len(p) - 1 for g, p in zip(group, self.paths)], [0] * pad]).astype(np.int64)
        fp8 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()  # noqa: E731
        self.ring = fp8(R, max(n_swa, 1), D)
        self.ring_pos = np.full((R, max(n_swa, 1)), -1, np.int64)
        for g in range(R):
            for p in range(max(0, self.pos0[g] - n_swa), self.pos0[g]):
                if n_swa and rng.random() < 0.9:
                    self.ring_pos[g, p % n_swa] = p
            if n_swa > 3 and g % 2:  # rows that dropped drafts of an earlier step left behind
                for p in range(self.pos0[g], self.pos0[g] + 3):
                    self.ring_pos[g, p % n_swa] = p
        self.draft = fp8(max(self.B, 1), D)
        self.weight = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if extras else None
        self.scaling = YARN if extras else None
        self.sink = (2 * rng.standard_normal(H)).astype(np.float32) if sink else None

    def seen(self, b):
        """(entry rows, ring rows, draft rows) of query b."""
        g, path = self.group[b], self.paths[b]
        e = list(range(self.n[g])) + ([self.n[g] + t for t in path] if self.entries else [])
        if not self.n_swa:
            return e, [], []
        p = self.q_pos[b]
        ring = [r for r in range(self.n_swa) if max(p - self.n_swa + 1, 0) <= self.ring_pos[g, r] < self.pos0[g]]
        return e, ring, [self.start[g] + t for t in path[max(0, len(path) - self.n_swa):]]

    def reference(self, of=None):
        res = []
        for b in range(self.B) if of is None else of:
            x = np.zeros((0, D))
            if b < len(self.group):
                e, ring, draft = self.seen(b)
                r = self.rows[self.group[b]][e]
                x = np.concatenate([decode(self.codes[r], self.scales[r]), F8[self.ring[self.group[b]][ring]], F8[self.draft[draft]]])
            q = self.q[b].double().numpy()
            if self.weight is not None:
                q = self.weight * q / np.sqrt((q ** 2).mean(-1, keepdims=True) + 1e-6)
                q = rotate(q[None], self.q_pos[b:b + 1], 64, 448, False, 10000.0, YARN)[0]
            o, lse, bound, lb = attention(x, q, SCALE, self.sink, self.weight is not None)
            if self.weight is not None:  # the output turns back: pairs mix
                o = rotate(o[None], self.q_pos[b:b + 1], 64, 448, False, 10000.0, YARN, inverse=True)[0]
                pair = bound[:, 448:].reshape(H, 32, 2).sum(-1, keepdims=True)
                top = np.abs(x).max() if len(x) else 0.0
                bound[:, 448:] = np.broadcast_to(pair, (H, 32, 2)).reshape(H, 64) + 2.0 ** -20 * top
            res.append((o, lse, bound, lb))
        return [np.stack(v) for v in zip(*res)]

    def device(self):
        t = {k: to_dev(getattr(self, k)) for k in ("codes", "scales", "table", "start", "parent", "q_pos", "ring", "ring_pos", "draft")}
        self.d = t
        N = self.n_pages * self.P
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.planes = csa2.Planes(t["codes"], t["scales"], torch.empty((N, 64), **u8), torch.empty((N, 4), **u8), self.P)
        self.pages = csa2.pages(t["table"], self.n_pages)
        self.dn, self.dq = to_dev(np.array(self.n, np.int32)), self.q.cuda()
        self.kw = dict(q_nr=csa2.norm_rope(to_dev(self.weight), 1e-6, True) if self.weight is not None else None,
                       scaling=csa2.rope_scaling(csa2.SCALE_YARN, *YARN[1:]) if self.scaling else None,
                       sink=to_dev(self.sink) if self.sink is not None else None)
        return self

    def workspace(self):
        ws = csa2.workspace(csa2.tree_attn_workspace_size(self.R, self.B, self.most, self.n_max, self.n_swa))
        ws.fill_(0xFF)
        return ws

    def run(self, dtype=torch.float32, ws=None, stream=None, out=None, lse=True):
        out = torch.full((self.B, H, D), 777.0, dtype=dtype, device="cuda") if out is None else out
        lse = torch.full((self.B, H), 777.0, device="cuda") if lse is True else lse
        ws = self.workspace() if ws is None else ws
        trees = csa2.trees(self.d["start"], self.d["parent"], self.R, self.B, self.most, self.entries)
        w = (self.d["ring"], self.d["ring_pos"], self.d["draft"]) if self.n_swa else (None, None, None)
        csa2.tree_attn_decode(self.planes, self.pages, trees, self.dn, self.n_max, *w, self.n_swa, self.dq, self.d["q_pos"], SCALE,
                              out, ws, lse_out=lse, stream=stream, **self.kw)
        return out, lse, ws

    def check(self, dtype=torch.float32, of=None, status=(0, 0), got=None):
        out, lse, ws = self.run(dtype) if got is None else got
        assert csa2.check(ws) == status
        close(out, lse, self.reference(of), of, dtype)
        return out, lse


def close(out, lse, ref, of, dtype):
    o, l, bound, lb = ref
    got = out.double().cpu().numpy()
    got_l = lse.double().cpu().numpy()
    if of is not None:
        got, got_l = got[of], got_l[of]
    off = np.abs(got - o)
    bound = bound + (np.abs(o) + bound) * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)
    assert (off <= bound).all(), (np.argwhere(off > bound)[:3], (off / np.maximum(bound, 1e-30)).max())
    none = np.isneginf(l)
    assert np.array_equal(np.isneginf(got_l), none)
    off = np.abs(got_l[~none] - l[~none])
    assert (off <= lb[~none]).all(), off.max()


SHAPES = {
    "one": ([9], [chain(1)]),
    "empty contexts": ([0, 0, 3], [chain(3), star(2), binary(5)]),
    "chain, star, binary": ([130, 64, 63], [chain(64), star(64), binary(64)]),
    "none drafted": ([40, 100, 7], [[], binary(9), []]),
    "ragged": ([200, 0, 1, 127, 128, 129, 500], [binary(7), chain(2), star(33), chain(1), [], binary(20), chain(31)]),
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("n_swa,entries", [(128, True), (0, True), (40, False), (5, True)])
def test_trees(shape, n_swa, entries, pairs, dtype):
    n, trees = SHAPES[shape]
    if pairs and sum(map(len, trees)) < 5 * len(n):
        trees = [t * 0 or random_tree(np.random.default_rng(len(t)), max(len(t), 9)) for t in trees]
    Forest(len(shape) + n_swa, n, trees, 16, n_swa, entries, pairs=pairs, sink=n_swa == 40, pad=n_swa % 3).device().check(dtype)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("P", [1, 7, 64, 100, 333])
def test_pages(P, pairs):
    rng = np.random.default_rng(P)
    Forest(P, [300, 17, 128], [random_tree(rng, 6), random_tree(rng, 5), random_tree(rng, 11)], P, 128, pairs=pairs).device().check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pairs", [False, True])
def test_norm_scaled_rotation_and_sink(pairs, dtype):
    rng = np.random.default_rng(1)
    trees = [random_tree(rng, T) for T in (13, 8, 1, 6)]
    Forest(7, [700, 256, 33, 0], trees, 32, 128, extras=True, sink=True, pad=2, pairs=pairs).device().check(dtype)


@pytest.mark.parametrize("seed", range(6))
def test_random_forests(seed):
    rng = np.random.default_rng(100 + seed)
    R = int(rng.integers(1, 12))
    trees = [random_tree(rng, int(rng.integers(0, 65))) for _ in range(R)]
    trees[0] = trees[0] or chain(5)
    n = rng.integers(0, 700, R).tolist()
    pairs = sum(map(len, trees)) >= 5 * R and seed % 2 == 0
    f = Forest(seed, n, trees, int(rng.integers(1, 80)), int(rng.choice([0, 3, 64, 128])), bool(rng.integers(0, 2)),
               bool(rng.integers(0, 2)), bool(rng.integers(0, 2)), int(rng.integers(0, 3)), pairs)
    f.device().check(torch.bfloat16 if seed % 3 else torch.float32)


def test_long_contexts():
    rng = np.random.default_rng(3)
    f = Forest(3, [12000, 4000], [random_tree(rng, 16), random_tree(rng, 12)], 64, 128)
    assert f.B ** 2 * f.n_max >= f.R << 21
    f.device().check(of=[0, 1, 7, 15, 16, 20, 27])


@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("n_swa,entries,extras,dtype", [(128, True, True, torch.bfloat16), (0, False, False, torch.float32)])
def test_bounds_that_cut_the_list(short, n_swa, entries, extras, dtype):
    # bounds of 20 requests of 6,000 entries make for a list in parts; the lengths fill all of them, or less than one
    rng = np.random.default_rng(23)
    R, bound = 20, 6000
    trees = [random_tree(rng, int(T)) for T in rng.integers(0, 40, R)]
    trees[0] = random_tree(rng, 40)
    n = rng.integers(0, 200 if short else bound, R)
    n[1], n[2] = 0, 200 if short else bound
    f = Forest(24, n.tolist(), trees, 64, n_swa, entries, extras, extras)
    f.n_max, narrow = bound, f.table
    f.max_pages = -(-(bound + csa2.MAX_TREE) // 64)
    f.table = np.full((R, f.max_pages), 0x7fffffff, np.int32)
    f.table[:, :narrow.shape[1]] = narrow
    assert R * -(-bound // 128) > 512 and f.B * bound // 256 >= 2 * 16 * 76
    of = sorted({0, f.B - 1, *rng.choice(f.B, 24, replace=False).tolist()})
    f.device().check(dtype, of=of)


def test_one_token_is_the_paged_attention():
    # a tree of one token: the same rows as csa2_paged_attn_decode over its context, itself and its window
    f = Forest(5, [333, 70], [chain(1), chain(1)], 16, 128).device()
    out, lse, _ = f.run()
    swa, pos = f.ring.copy(), np.where(f.ring_pos < f.pos0[:, None], f.ring_pos, -1)
    for g in range(2):  # the token's own window row in its place of the ring
        swa[g, f.pos0[g] % 128], pos[g, f.pos0[g] % 128] = f.draft[g], f.pos0[g]
    other, other_lse = torch.empty_like(out), torch.empty_like(lse)
    ws = csa2.workspace(csa2.paged_attn_workspace_size(2, 400, 128))
    win = csa2.window(to_dev(pos), to_dev(f.q_pos - 127))
    csa2.paged_attn_decode(f.planes, f.pages, 2, to_dev(np.array([334, 71], np.int32)), 334, to_dev(swa), 128, f.dq, SCALE, other, ws,
                           lse_out=other_lse, win=win)
    bound = f.reference()[2]
    assert (np.abs((out - other).double().cpu().numpy()) <= 2 * bound).all()
    assert (lse - other_lse).abs().max() <= 2.0 ** -12


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("what", ["entry", "draft", "ring", "context"])
def test_nan_reaches_those_that_see_it(what, pairs):
    tree = [-1, 0, 0, 1, 1, 2, -1, 6, 3]
    f = Forest(6, [140, 90], [tree, tree], 16, 128, pairs=pairs)
    if what == "entry":
        f.scales[f.rows[0][140 + 1], 5] = 0xFF
        hit = [t for t in range(9) if 1 in path_to(tree, t)]
    elif what == "draft":
        f.draft[f.start[1] + 2, 17] = 0x7F
        hit = [9 + t for t in range(9) if 2 in path_to(tree, t)]
    elif what == "ring":
        f.pos0[0], f.ring_pos[0] = 300, -1
        f.q_pos[:9] = [300 + len(path_to(tree, t)) - 1 for t in range(9)]
        f.ring_pos[0, 174 % 128] = 174  # in the window of depth 0 and 1 alone
        f.ring[0, 174 % 128, 0] = 0x7F
        hit = [t for t in range(9) if len(path_to(tree, t)) <= 2]
    else:
        f.scales[f.rows[1][3], 0] = 0x7F
        hit = list(range(9, 18))
    out, lse, ws = f.device().run()
    assert csa2.check(ws) == (0, 0)
    bad = out.isnan().flatten(1).all(1)
    assert bad.nonzero().flatten().tolist() == hit and not out[~bad].isnan().any()
    rest = [b for b in range(18) if b not in hit]
    close(out, lse, f.reference(rest), rest, torch.float32)


@pytest.mark.parametrize("pairs", [False, True])
def test_bad_parents_count_as_roots_and_are_reported(pairs):
    tree = [-1, 0, 0, 1, 4, 2, 99, -2]
    as_roots = [-1, 0, 0, 1, -1, 2, -1, -1]
    f = Forest(8, [100], [as_roots], 16, 128, pairs=pairs)
    f.parent[:8] = tree
    out, lse, ws = f.device().run()
    status, detail = csa2.check(ws)
    assert status == 6 and detail in (4, 6, 7)
    close(out, lse, f.reference(), None, torch.float32)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("start", [[0, 9, 5], [-1, 3, 18], [0, 9, 99], [10, 12, 13]])
def test_starts_out_of_order(start, pairs):
    f = Forest(9, [100, 50], [star(9), star(9)], 16, 128, sink=True, pairs=pairs).device()
    ordered = start == [10, 12, 13]  # queries before and behind the trees see nothing
    f.d["start"].copy_(to_dev(np.array(start, np.int32)))
    out, lse, ws = f.run()
    assert csa2.check(ws)[0] == (0 if ordered else 6)
    none = [b for b in range(18) if not ordered or not 10 <= b < 13]
    # the logit goes to log2 units and back: two roundings of 2^-24, and the constant's
    assert (out[none] == 0).all() and ((lse[none] - f.kw["sink"]).abs() <= 2.0 ** -22 * f.kw["sink"].abs()).all()


def test_trees_beyond_the_bound_and_contexts_beyond_theirs():
    f = Forest(10, [100, 50], [binary(9), binary(6)], 16, 128).device()
    f.most = 8
    out, lse, ws = f.run()
    assert csa2.check(ws) == (6, 0) and (out == 0).all() and lse.isneginf().all()
    f = Forest(10, [100, 50], [binary(9), binary(6)], 16, 0, entries=False).device()
    want = f.run()[0]
    f.dn.copy_(to_dev(np.array([1 << 30, -5], np.int32)))  # counts as n_max, and as none
    out, lse, ws = f.run()
    assert csa2.check(ws) == (0, 0)
    assert torch.equal(out[:9], want[:9]) and (out[9:] == 0).all() and lse[9:].isneginf().all()


@pytest.mark.parametrize("pairs", [False, True])
def test_bad_pages_are_skipped_and_reported(pairs):
    f = Forest(11, [100, 50], [binary(9), binary(6)], 16, 128, pairs=pairs).device()
    for page in (-1, f.n_pages, 0x7fffffff):
        f.d["table"][1, 1] = page
        out, lse, ws = f.run()
        assert csa2.check(ws) == (6, page)
        keep = np.r_[0:16, 32:f.n[1] + 6]
        g = Forest(11, [100, 50], [binary(9), binary(6)], 16, 128, pairs=pairs)
        g.n[1] -= 16
        g.rows[1] = f.rows[1][keep]
        close(out, lse, g.reference(), None, torch.float32)


def test_no_window_rows_and_no_context_gives_zero():
    f = Forest(12, [0], [binary(5)], 16, 0, entries=False).device()
    out, lse, ws = f.run(torch.bfloat16)
    assert csa2.check(ws) == (0, 0) and (out == 0).all() and lse.isneginf().all()


def test_same_bits_again_without_lse_and_on_another_stream():
    f = Forest(13, [2000, 900], [binary(40), chain(30)], 64, 128, extras=True, pairs=True).device()
    out, lse, _ = f.run(torch.bfloat16)
    side = torch.cuda.Stream()
    ws = f.workspace()
    side.wait_stream(torch.cuda.current_stream())
    again = torch.empty_like(out)
    f.run(torch.bfloat16, ws=ws, stream=side, out=again, lse=None)
    side.synchronize()
    assert torch.equal(out, again)
    # two calls at once, each with its own workspace
    a, b, wa, wb = torch.empty_like(out), torch.empty_like(out), f.workspace(), f.workspace()
    torch.cuda.synchronize()
    f.run(torch.bfloat16, ws=wa, stream=side, out=a, lse=None)
    f.run(torch.bfloat16, ws=wb, out=b, lse=None)
    torch.cuda.synchronize()
    assert torch.equal(out, a) and torch.equal(out, b)


@pytest.mark.parametrize("pairs", [False, True])
def test_graph_replayed_on_other_trees(pairs):
    rng = np.random.default_rng(14)
    f = Forest(14, [300, 200, 100], [random_tree(rng, 10) for _ in range(3)], 16, 128, pairs=pairs, pad=3).device()
    f.most = csa2.MAX_TREE
    out, lse = torch.empty((f.B, H, D), device="cuda"), torch.empty((f.B, H), device="cuda")
    ws = f.workspace()
    f.run(ws=ws, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.run(ws=ws, out=out, lse=lse)
    # other lengths and trees of as many queries in the same buffers
    g = Forest(15, [250, 200, 7], [random_tree(rng, 6), random_tree(rng, 13), random_tree(rng, 11)], 16, 128, pairs=pairs, pad=3)
    g.codes, g.scales = f.codes.copy(), f.scales.copy()
    g.table, g.rows = f.table, []
    total = [h + len(t) for h, t in zip(g.n, g.trees)]
    for r in range(3):
        e = np.arange(min(total[r], f.n[r] + 10))
        g.rows.append(f.table[r, e // 16].astype(np.int64) * 16 + e % 16)
    g.n[1] = 197  # its pages hold 210 entries
    for k in ("start", "parent", "q_pos", "ring", "ring_pos", "draft"):
        f.d[k].copy_(to_dev(getattr(g, k)))
    f.dq.copy_(g.q.cuda())
    f.dn.copy_(to_dev(np.array(g.n, np.int32)))
    graph.replay()
    assert csa2.check(ws) == (0, 0)
    close(out, lse, g.reference(), None, torch.float32)


@pytest.mark.parametrize("pairs", [False, True])
def test_more_requests_than_the_plans_lists_hold(pairs):
    # lists of 2,048 requests and more lie in global memory, and those of 4,096 pairs and more
    R = 2100 if pairs else 5000
    rng = np.random.default_rng(16)
    trees = [binary(int(T)) for T in (rng.integers(4, 9, R) if pairs else rng.integers(0, 3, R))]
    trees[0], trees[-1] = binary(9), binary(9)
    f = Forest(16, rng.integers(0, 30, R).tolist(), trees, 16, 3, pairs=pairs)
    assert not pairs or (f.B > 8400 and f.B ** 2 * f.n_max >= R << 21)
    f.device().check(torch.bfloat16, of=[0, 5, 8, 9, f.B // 3, f.B // 2, f.B - 9, f.B - 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("extras,sink", [(True, True), (True, False), (False, True), (False, False)])
def test_more_pairs_than_parts(extras, sink, dtype):
    # most pairs are one CTA pair's as a whole
    R = 90
    rng = np.random.default_rng(17 + extras)
    trees = [random_tree(rng, int(T)) for T in rng.integers(3, 12, R)]
    trees[3], trees[40], trees[-1] = [], chain(11), star(1)
    f = Forest(17, rng.integers(0, 60, R).tolist(), trees, 16, 128, extras=extras, sink=sink, pairs=True, pad=2)
    f.device()
    out, lse = f.check(dtype, of=sorted(rng.choice(f.B, 60, replace=False).tolist()) + [f.B - 3, f.B - 1])
    # without the logsumexp the same outputs
    again, _, ws = f.run(dtype, lse=None)
    assert csa2.check(ws) == (0, 0) and torch.equal(out, again)
