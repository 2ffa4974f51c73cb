"""csa2_tree_commit against Python lists: entries of accepted paths, window rows, what stays as it was, refusals that
are found on the device."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Case:
    def __init__(self, seed, have, tokens, paths, P, n_win=128, entries=True, n_path=None, max_tokens=64, pos=None):
        rng = np.random.default_rng(seed)
        R = self.R = len(have)
        self.have, self.tokens, self.paths, self.P, self.n_win, self.entries = have, tokens, paths, P, n_win, entries
        self.max_tokens = max_tokens
        self.start = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
        self.B = int(self.start[-1])
        total = [h + t for h, t in zip(have, tokens)]
        self.max_pages = max(1, max(-(-t // P) for t in total))
        self.n_pages = sum(-(-t // P) for t in total) + 2
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((R, self.max_pages), 0x7fffffff, np.int32)
        at = 0
        for g, t in enumerate(total):
            n = -(-t // P)
            self.table[g, :n] = ids[at:at + n]
            at += n
        N = self.n_pages * P
        self.parts = [rng.integers(0, 256, (N, w)).astype(np.uint8) for w in (256, 32, 64, 4)]
        self.n_path = n_path if n_path is not None else max([1] + [len(p) for p in paths])
        self.path = np.full((R, self.n_path), -77, np.int32)  # behind a path: not read
        for g, p in enumerate(paths):
            self.path[g, :len(p)] = p[:self.n_path]
        self.accept = np.array([len(p) for p in paths], np.int32)
        self.draft = rng.integers(0, 256, (max(self.B, 1), 512)).astype(np.uint8)
        self.ring = rng.integers(0, 256, (R, max(n_win, 1), 512)).astype(np.uint8)
        self.ring_pos = rng.integers(-1, 1000, (R, max(n_win, 1))).astype(np.int64)
        self.pos = np.array([1000 + 37 * g for g in range(R)] if pos is None else pos, np.int64)

    def row(self, g, e):
        return self.table[g, e // self.P] * self.P + e % self.P

    def expected(self, skip=()):
        parts, ring, ring_pos = [p.copy() for p in self.parts], self.ring.copy(), self.ring_pos.copy()
        new = []
        for g, p in enumerate(self.paths):
            if g in skip:
                new.append(0)
                continue
            new.append(len(p) - self.tokens[g] if self.entries else 0)
            if self.entries:
                for old, now in zip(self.parts, parts):
                    for i, t in enumerate(p):
                        now[self.row(g, self.have[g] + i)] = old[self.row(g, self.have[g] + t)]
            for i, t in enumerate(p):
                if self.n_win:
                    at = (self.pos[g] + i) % self.n_win
                    ring[g, at], ring_pos[g, at] = self.draft[self.start[g] + t], self.pos[g] + i
        return parts, ring, ring_pos, new

    def run(self, stream=None, **put):
        d = {k: to_dev(np.asarray(put.get(k, getattr(self, k)))) for k in
             ("start", "table", "path", "accept", "draft", "ring", "ring_pos", "pos")}
        self.dev = parts = [to_dev(p) for p in self.parts]
        have = to_dev(np.array(put.get("have", self.have), np.int32))
        new = torch.full((self.R,), 777, dtype=torch.int32, device="cuda")
        ws = csa2.workspace(csa2.tree_commit_workspace_size(self.R))
        ws.fill_(0xFF)
        trees = csa2.trees(d["start"], None, self.R, self.B, self.max_tokens, self.entries)
        planes = csa2.Planes(*parts, self.P) if self.entries else None
        pages = csa2.pages(d["table"], put.get("n_pages", self.n_pages)) if self.entries else None
        win = dict(draft=d["draft"], pos=d["pos"], ring=d["ring"], ring_pos=d["ring_pos"], n_win=self.n_win) if self.n_win else {}
        self.call = lambda **kw: csa2.tree_commit(planes, pages, trees, have if self.entries else None, d["accept"],  # noqa: E731
                                                  d["path"], self.n_path, new, ws, **win, **kw)
        self.d, self.new, self.ws = d, new, ws
        self.call(stream=stream)
        status = csa2.check(ws)
        return status, [p.cpu().numpy() for p in parts], d["ring"].cpu().numpy(), d["ring_pos"].cpu().numpy(), new.tolist()

    def check(self, skip=(), status=(0, 0), **put):
        got, want = self.run(**put), self.expected(skip)
        assert got[0] == status
        for a, b in zip(got[1], want[0]):
            assert np.array_equal(a, b)
        assert np.array_equal(got[2], want[1]) and np.array_equal(got[3], want[2]) and got[4] == want[3]


@pytest.mark.parametrize("P", [1, 7, 16, 64])
@pytest.mark.parametrize("n_win", [0, 5, 128])
def test_paths(P, n_win):
    paths = [[0, 1, 2], [1, 4, 5, 9], [], [63], list(range(64)), [0], [], list(range(0, 64, 2)), [3, 1, 2], [2, 2, 0]]
    tokens = [8, 10, 5, 64, 64, 1, 0, 64, 4, 3]
    Case(P + n_win, [0, 5, 100, 64, 17, 3, 9, 128, 1, 62], tokens, paths, P, n_win).check()


def test_without_entries():
    Case(1, [5, 9], [6, 3], [[0, 2, 5], [1]], 16, entries=False).check()


@pytest.mark.parametrize("R", [1, 300])
def test_many_requests(R):
    rng = np.random.default_rng(R)
    tokens = rng.integers(0, 65, R).tolist()
    paths = [sorted(rng.permutation(t)[:rng.integers(0, t + 1)].tolist()) for t in tokens]
    Case(R, rng.integers(0, 90, R).tolist(), tokens, paths, 16).check()


def test_far_positions():
    Case(2, [4, 5], [3, 4], [[0, 2], [1, 3]], 8, pos=[(1 << 40) + 3, 0]).check()


@pytest.mark.parametrize("put,skip", [
    (dict(accept=[2, 5]), 1), (dict(accept=[-1, 1]), 0), (dict(accept=[4, 1]), 0), (dict(path=[[0, 3, 0], [1, 0, 0]]), 0),
    (dict(path=[[0, -1, 0], [1, 0, 0]]), 0), (dict(start=[0, 3, 99]), 1), (dict(start=[4, 3, 7]), 0), (dict(start=[-1, 3, 7]), 0),
    (dict(have=[4, -1]), 1), (dict(have=[4, 1 << 30]), 1), (dict(pos=[-1, 5]), 0),
    (dict(pos=[3, (1 << 63) - 2]), 1)])
def test_what_is_out_of_range_stays_as_it_is(put, skip):
    c = Case(3, [4, 5], [3, 4], [[0, 2], [1]], 8, n_path=3)
    put = {k: np.array(v, np.int64 if k == "pos" else np.int32) for k, v in put.items()}
    if "start" in put and skip == 0:  # the second request is as it was
        assert put["start"][1] == 3
    if "start" in put and skip == 1:
        put["start"] = put["start"].astype(np.int32)
    pos = put.get("pos")
    if pos is not None:
        c.pos = pos.copy()
    c.check(skip=(skip,), status=(6, skip), **put)


def test_pages_outside_the_planes():
    c = Case(4, [4, 5], [3, 4], [[0, 2], [1]], 8, n_path=3)
    c.check(skip=(0,), status=(6, 0), table=np.where(np.arange(2)[:, None] == 0, c.n_pages, c.table).astype(np.int32))
    c.check(skip=(1,), status=(6, 1), table=np.where(np.arange(2)[:, None] == 1, -1, c.table).astype(np.int32))


def test_trees_beyond_the_bound():
    Case(5, [4, 5], [3, 4], [[0, 2], [1]], 8, n_path=3, max_tokens=3).check(skip=(1,), status=(6, 1))


def test_stream_and_graph():
    c = Case(6, [4, 5, 64], [3, 4, 30], [[0, 2], [1], [3, 9, 29]], 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = c.run(stream=side)
    want = c.expected()
    assert got[0] == (0, 0) and all(np.array_equal(a, b) for a, b in zip(got[1], want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for t, p in zip(c.dev, c.parts):
        t.copy_(to_dev(p))
    c.d["ring"].copy_(to_dev(c.ring))
    c.d["ring_pos"].copy_(to_dev(c.ring_pos))
    graph.replay()
    assert csa2.check(c.ws) == (0, 0)
    assert all(np.array_equal(t.cpu().numpy(), b) for t, b in zip(c.dev, want[0]))
    assert np.array_equal(c.d["ring"].cpu().numpy(), want[1])
