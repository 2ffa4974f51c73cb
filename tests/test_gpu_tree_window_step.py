"""Serving steps with draft trees as in test_gpu_tree_step, whose window rows are normalised and rotated on the way into
the drafts' rows and the ring (csa2_swa_append), as the queries and entries are; no scaling, which the window's rotation
does not have."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from paged_common import F8, H, attention, decode
from rotary_common import rotate
from test_gpu_tree_step import SCALE, WIN, Server

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class WindowServer(Server):
    def __init__(self, *args):
        super().__init__(*args)
        self.sc, self.rot = None, csa2.rotary(64, 0, csa2.ROPE_HALVES)
        self.zero = self.pos  # a draft's window row is its only one: place pos mod 1, rotated by pos

    def normalised(self, x, pos):
        y = self.weight.cpu().double().numpy() * x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6)
        return rotate(y, pos, 64, 448, False, 10000.0)

    def window(self, x, pos):
        """Window rows of latents x at pos: the append's bytes, each E4M3's nearest to the definition's value."""
        n = len(x)
        rows = torch.zeros(n, 1, 512, dtype=torch.uint8, device="cuda")
        csa2.swa_append(to_dev(x), n, to_dev(pos), n, rows, 1)
        got, y = F8[rows.cpu().numpy()[:, 0]], self.normalised(x.astype(np.float64), pos)
        # half a step (2^-4 of the value, 2^-10 below 2^-6) and the fp32 of norm and rotation, 2^-18 of the largest
        assert (np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + 2.0 ** -18 * np.abs(y).max()).all()
        return got

    def check(self, n, group, paths, x):
        codes, scales = self.planes.kv_codes.cpu().numpy(), self.planes.kv_scales.cpu().numpy()
        first = self.start.tolist()
        for b in {0, n // 2, n - 1} if n else ():
            g, path, have = group[b], paths[b], len(self.tokens[group[b]])
            at = self.rows(g, have + max(path) + 1)[list(range(have)) + [have + t for t in path]]
            seen = np.array([t[0] for t in self.tokens[g]] + [x[first[g] + t] for t in path], np.float32)
            p = np.arange(len(seen))[-WIN:]
            rows = np.concatenate([decode(codes[at], scales[at]), self.window(seen[-WIN:], p)])
            p = self.pos[b:b + 1].cpu().numpy()
            q = self.normalised(self.q[b].cpu().double().numpy()[None], p)[0]
            o, lse, bound, lb = attention(rows, q, SCALE, q_rounded=True)
            o = rotate(o[None], p, 64, 448, False, 10000.0, inverse=True)[0]
            pair = bound[:, 448:].reshape(H, 32, 2).sum(-1, keepdims=True)
            bound[:, 448:] = np.broadcast_to(pair, (H, 32, 2)).reshape(H, 64) + 2.0 ** -20 * np.abs(rows).max()
            bound += (np.abs(o) + bound) * 2.0 ** -24
            assert (np.abs(self.out[b].cpu().double().numpy() - o) <= bound).all()
            assert (np.abs(self.lse[b].cpu().double().numpy() - lse) <= lb).all()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("R,most,P", [(3, 9, 4), (2, 24, 16)])
def test_steps(R, most, P, graph, monkeypatch):
    s = WindowServer(40 + R, R, most, P, graph)
    plain = csa2.swa_append
    monkeypatch.setattr(csa2, "swa_append", lambda *a, **k: plain(*a, nr=s.nr, **k))
    for _ in range(7):
        if max(len(t) for t in s.tokens) > s.n_max:
            break
        s.step()
    s.check_cache()  # the ring too is that of the accepted tokens, normalised and rotated
    assert sum(map(len, s.tokens)) > 0
