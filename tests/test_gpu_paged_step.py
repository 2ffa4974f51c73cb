"""Serving steps over a paged cache as a loop runs them: page tables, appends, window and attention of one fixed
size, padded, captured once and replayed."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from paged_common import D, F8, H, PagedState, attention, decode

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("m", [1, 2])
def test_padded_rows_are_skipped_without_a_report(m):
    d, G, n_slots, P = 128, 5, 3, 16
    rng = np.random.default_rng(m)
    w = [to_dev(rng.standard_normal(s).astype(np.float32) * d ** -0.5).to(torch.bfloat16)
         for s in ((d, 512), (d, 512), (512, 128))]
    hidden = to_dev(rng.standard_normal((G, m, d)).astype(np.float32)).to(torch.bfloat16)
    ws = csa2.workspace(csa2.cache_append_workspace_size(G, d, m))
    slots, entries = np.array([1, -1, 2, -1, 0], np.int32), np.array([3, -1, 15, -1, 7], np.int64)

    def append(s, e):
        planes = csa2.Planes.empty(n_slots, P)
        parts = (planes.kv_codes, planes.kv_scales, planes.ix_codes, planes.ix_scales)
        for t in parts:
            t.fill_(0xA5)
        csa2.cache_append(hidden, G, d, *w, m, planes, n_slots, to_dev(s), to_dev(e), ws)
        return csa2.check(ws), parts

    status, got = append(slots, entries)
    assert status == (0, 0)
    full, want = append(np.where(slots < 0, 2, slots).astype(np.int32), np.where(entries < 0, [0, 1, 0, 4, 0], entries))
    assert full == (0, 0)
    rows = [P + 3, 2 * P + 15, 7]
    for a, b in zip(got, want):
        assert torch.equal(a[rows], b[rows])
        rest = np.setdiff1d(np.arange(n_slots * P), rows)
        assert (a[rest] == 0xA5).all()
    # anything else outside the planes is still reported, beside padding too
    for s, e, detail in ((-1, 3, -1), (1, -1, -1), (-2, -1, -2), (3, 0, 3), (0, P, P)):
        slots[3], entries[3] = s, e
        assert append(slots, entries)[0] == (6, detail)


@pytest.mark.parametrize("n_win", [8, 128])
@pytest.mark.parametrize("nr", [False, True])
def test_of_more_rows_than_the_ring_the_last_are_kept(n_win, nr):
    # chunks of a prefill: several times the ring, once as many rows, fewer, and none; padding behind them
    count, first = [5 * n_win + 3, n_win, 3, 0, n_win + 1], [1000, 17, n_win - 1, 0, 1 << 33]
    query = np.concatenate([np.full(c, b) for b, c in enumerate(count)] + [[-1] * 2]).astype(np.int32)
    pos = np.concatenate([f + np.arange(c) for f, c in zip(first, count)] + [[-1] * 2]).astype(np.int64)
    R, B = len(pos), len(count)
    x = to_dev(np.random.default_rng(n_win).standard_normal((R, 512)).astype(np.float32))
    kw = dict(nr=csa2.norm_rope(None, 1e-6, True)) if nr else {}
    last = np.concatenate([np.flatnonzero(query == b)[-n_win:] for b in range(B)])
    rings = []
    for rows in (np.arange(R), last):  # all rows, and the last ones alone
        ring = torch.full((B, n_win, 512), 0xA5, dtype=torch.uint8, device="cuda")
        at = torch.full((B, n_win), -1, dtype=torch.int64, device="cuda")
        csa2.swa_append(x[torch.from_numpy(rows).cuda()], len(rows), to_dev(pos[rows]), B, ring, n_win,
                        query=to_dev(query[rows]), ring_pos=at, **kw)
        rings.append((ring, at))
    assert torch.equal(rings[0][0], rings[1][0]) and torch.equal(rings[0][1], rings[1][1])
    for b in range(B):
        kept = set(range(first[b] + max(count[b] - n_win, 0), first[b] + count[b]))
        assert set(rings[0][1][b].tolist()) - {-1} == kept
