"""Serving steps with draft trees as a loop runs them: page tables grow by the drafts, their latents are appended
with norm and scaled rotation, the tree attention verifies them, the accepted path is committed and the rest dropped.  After
several steps cache and ring are those of a request that only ever saw the accepted tokens."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from paged_common import D, F8, H, attention, decode
from rotary_common import rotate

pytestmark = pytest.mark.gpu
SCALE, WIN, YARN = 512 ** -0.5, 16, ("yarn", 4.0, 4096, 32.0, 1.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def path_to(parents, t):
    out = []
    while t >= 0:
        out.insert(0, t)
        t = parents[t]
    return out


class Server:
    """Buffers of fixed sizes: R requests, up to B drafted tokens a step, P entries a page."""

    def __init__(self, seed, R, most, P, graph):
        rng = np.random.default_rng(seed)
        self.rng, self.R, self.B, self.most, self.P, self.graph = rng, R, R * most, most, P, graph
        self.max_pages, self.n_pages = 12, 12 * R
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        i64 = lambda *s: torch.zeros(s, dtype=torch.int64, device="cuda")  # noqa: E731
        u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
        B = self.B
        self.planes = csa2.Planes.empty(self.n_pages, P)
        for t in (self.planes.kv_codes, self.planes.ix_codes, self.planes.ix_scales):
            t.zero_()
        self.planes.kv_scales.fill_(0x7F)  # what nothing has written is NaN
        self.table, self.free = i32(R, self.max_pages).fill_(-1), i32(self.n_pages)
        self.free.copy_(to_dev(rng.permutation(self.n_pages).astype(np.int32)))
        self.n_free, self.have, self.new = i32(1).fill_(self.n_pages), i32(R), i32(R)
        self.total, self.drop, self.start = i32(R), i32(R), i32(R + 1)
        self.slot, self.entry = i32(B), i64(B)
        self.parent, self.pos, self.x, self.key = i32(B), i64(B), torch.zeros(B, D, device="cuda"), torch.zeros(B, 128, device="cuda")
        self.draft, self.zero = u8(B, D), i64(B)
        self.ring, self.ring_pos = u8(R, WIN, D), i64(R, WIN).fill_(-1)
        self.q, self.out, self.lse = torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, H, D, device="cuda"), torch.zeros(B, H, device="cuda")
        self.accept, self.path, self.pos0 = i32(R), i32(R, most), i64(R)
        self.weight = to_dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32))
        self.nr, self.sc = csa2.norm_rope(self.weight, 1e-6, True), csa2.rope_scaling(csa2.SCALE_YARN, *YARN[1:])
        self.rot = csa2.rotary(64, 0, csa2.ROPE_HALVES, scaling=self.sc)
        self.pages = csa2.pages(self.table, self.n_pages)
        self.trees = csa2.trees(self.start, self.parent, R, B, most)
        self.n_max = self.max_pages * P - most
        self.ws = [csa2.workspace(n) for n in (csa2.page_tables_workspace_size(R), csa2.latent_append_workspace_size(B),
                                               csa2.tree_attn_workspace_size(R, B, most, self.n_max, WIN),
                                               csa2.tree_commit_workspace_size(R), csa2.page_tables_workspace_size(R))]
        self.runs = {}
        # per request: the accepted tokens' latents and keys
        self.tokens = [[] for _ in range(R)]

    def verify(self):
        w = self.ws
        # the contexts stay in `have`; `total` has the drafts too
        csa2.page_tables(self.R, self.have, self.new, self.P, self.table, self.max_pages, self.n_pages, self.free, self.n_free,
                         self.n_free, self.total, w[0], n_rows=self.B, slot=self.slot, entry=self.entry, row_start=self.start)
        csa2.latent_append(self.x, self.B, self.planes, self.n_pages, self.slot, self.entry, w[1], key=self.key, kv_nr=self.nr,
                           scaling=self.sc, pos=self.pos, key_rot=self.rot)
        csa2.swa_append(self.x, self.B, self.zero, self.B, self.draft, 1)  # a window row for every draft
        csa2.tree_attn_decode(self.planes, self.pages, self.trees, self.have, self.n_max, self.ring, self.ring_pos, self.draft, WIN,
                              self.q, self.pos, SCALE, self.out, w[2], lse_out=self.lse, q_nr=self.nr, scaling=self.sc)

    def commit(self):
        csa2.tree_commit(self.planes, self.pages, self.trees, self.have, self.accept, self.path, self.most, self.drop, self.ws[3],
                         draft=self.draft, pos=self.pos0, ring=self.ring, ring_pos=self.ring_pos, n_win=WIN)
        csa2.page_tables(self.R, self.total, self.drop, self.P, self.table, self.max_pages, self.n_pages, self.free, self.n_free,
                         self.n_free, self.have, self.ws[4])

    def run(self, what):
        if not self.graph:
            return getattr(self, what)()
        if what not in self.runs:  # captured once, after an eager step
            getattr(self, what)()
            self.runs[what] = None
            return
        if self.runs[what] is None:
            self.runs[what] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.runs[what]):
                getattr(self, what)()
        self.runs[what].replay()

    def step(self):
        rng, R = self.rng, self.R
        parents = [[-1 if t == 0 or rng.random() < 0.2 else int(rng.integers(0, t)) for t in range(rng.integers(0, self.most + 1))]
                   for _ in range(R)]
        T = [len(p) for p in parents]
        have = [len(t) for t in self.tokens]
        paths = [path_to(p, i) for p in parents for i in range(len(p))]
        group = np.repeat(np.arange(R), T)
        n = sum(T)
        x, key, pos = np.zeros((self.B, D), np.float32), np.zeros((self.B, 128), np.float32), np.zeros(self.B, np.int64)
        x[:n], key[:n] = rng.standard_normal((n, D)), rng.standard_normal((n, 128))
        pos[:n] = [have[g] + len(p) - 1 for g, p in zip(group, paths)]
        for t, v in ((self.x, x), (self.key, key), (self.pos, pos), (self.new, np.array(T, np.int32)),
                     (self.pos0, np.array(have, np.int64)),
                     (self.parent, np.array([p for t in parents for p in t] + [0] * (self.B - n), np.int32))):
            t.copy_(to_dev(v))
        self.q.copy_(to_dev(rng.standard_normal((self.B, H, D)).astype(np.float32)).to(torch.bfloat16))
        self.run("verify")
        assert [csa2.check(w)[0] for w in self.ws[:3]] == [0, 0, 0]
        assert self.start.tolist() == np.concatenate([[0], np.cumsum(T)]).tolist() and self.have.tolist() == have
        self.check(n, group, paths, x)
        # a random leaf's path, or a part of it, is accepted
        accept, path = np.zeros(R, np.int32), np.full((R, self.most), -1, np.int32)
        at = 0
        for g in range(R):
            if T[g]:
                p = path_to(parents[g], int(rng.integers(0, T[g])))
                p = p[:int(rng.integers(0, len(p) + 1))]
                accept[g], path[g, :len(p)] = len(p), p
                self.tokens[g] += [(x[at + t], key[at + t]) for t in p]
            at += T[g]
        self.accept.copy_(to_dev(accept))
        self.path.copy_(to_dev(path))
        self.run("commit")
        assert csa2.check(self.ws[3]) == (0, 0) and csa2.check(self.ws[4]) == (0, 0)
        assert self.have.tolist() == [len(t) for t in self.tokens]

    def rows(self, g, n):
        e = np.arange(n)
        return self.table.cpu().numpy()[g, e // self.P].astype(np.int64) * self.P + e % self.P if n else np.zeros(0, np.int64)

    def check(self, n, group, paths, x):
        codes, scales = self.planes.kv_codes.cpu().numpy(), self.planes.kv_scales.cpu().numpy()
        first = self.start.tolist()
        weight = self.weight.cpu().numpy()
        for b in {0, n // 3, n // 2, n - 1} if n else ():
            g, path, have = group[b], paths[b], len(self.tokens[group[b]])
            at = self.rows(g, have + max(path) + 1)[list(range(have)) + [have + t for t in path]]
            # the window: the last WIN tokens of context and path
            window = np.array([t[0] for t in self.tokens[g]] + [x[first[g] + t] for t in path], np.float32)[-WIN:]
            window = F8[torch.from_numpy(window).to(torch.float8_e4m3fn).view(torch.uint8).numpy()]
            p = self.pos[b:b + 1].cpu().numpy()
            q = self.q[b].cpu().double().numpy()
            q = weight * q / np.sqrt((q ** 2).mean(-1, keepdims=True) + 1e-6)
            q = rotate(q[None], p, 64, 448, False, 10000.0, YARN)[0]
            rows = np.concatenate([decode(codes[at], scales[at]), window])
            o, lse, bound, lb = attention(rows, q, SCALE, q_rounded=True)
            o = rotate(o[None], p, 64, 448, False, 10000.0, YARN, inverse=True)[0]
            pair = bound[:, 448:].reshape(H, 32, 2).sum(-1, keepdims=True)
            bound[:, 448:] = np.broadcast_to(pair, (H, 32, 2)).reshape(H, 64) + 2.0 ** -20 * np.abs(rows).max()
            bound += (np.abs(o) + bound) * 2.0 ** -24
            assert (np.abs(self.out[b].cpu().double().numpy() - o) <= bound).all()
            assert (np.abs(self.lse[b].cpu().double().numpy() - lse) <= lb).all()

    def check_cache(self):
        """The accepted tokens appended at once to another cache give the same bytes, and their last window rows the ring."""
        for g, tokens in enumerate(self.tokens):
            n = len(tokens)
            if not n:
                continue
            x, key = (to_dev(np.array([t[i] for t in tokens], np.float32)) for i in (0, 1))
            other = csa2.Planes.empty(1, n)
            e, ws = torch.arange(n, device="cuda"), csa2.workspace(256)
            csa2.latent_append(x, n, other, 1, torch.zeros(n, dtype=torch.int32, device="cuda"), e, ws, key=key, kv_nr=self.nr,
                               scaling=self.sc, pos=e, key_rot=self.rot)
            at = torch.from_numpy(self.rows(g, n)).cuda()
            for name in ("kv_codes", "kv_scales", "ix_codes", "ix_scales"):
                assert torch.equal(getattr(self.planes, name)[at], getattr(other, name)), name
            ring = torch.zeros(1, WIN, D, dtype=torch.uint8, device="cuda")
            where = torch.full((1, WIN), -1, dtype=torch.int64, device="cuda")
            csa2.swa_append(x, n, e, 1, ring, WIN, query=torch.zeros(n, dtype=torch.int32, device="cuda"), ring_pos=where)
            assert torch.equal(self.ring_pos[g], where[0]) and torch.equal(self.ring[g], ring[0])
        used = sum(-(-len(t) // self.P) for t in self.tokens)
        assert self.n_free.item() == self.n_pages - used


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("R,most,P", [(3, 9, 4), (5, 16, 16), (1, 40, 32)])
def test_steps(R, most, P, graph):
    s = Server(R, R, most, P, graph)
    for _ in range(9):
        if max(len(t) for t in s.tokens) > s.n_max:
            break
        s.step()
    s.check_cache()
    assert sum(map(len, s.tokens)) > 0
