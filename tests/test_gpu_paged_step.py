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


def test_a_request_that_fell_into_its_kept_pages_grows_in_pages_of_its_own():
    # two requests on two full shared pages; request 0 drops 100 of 128 entries and grows again
    P, kept = 64, np.array([2, 2], np.int32)
    s = PagedState(2, P, 4, 10, [9, 8, 7, 6, 5])
    s.have = [128, 200]
    s.table[0][:2], s.table[1][:4] = [0, 1], [0, 1, 2, 3]
    i32 = lambda v: to_dev(np.asarray(v, np.int32))
    have, table, free, n_free = i32(s.have), i32(s.table), i32(s.free), i32([s.n_free])
    e = lambda n, t: torch.empty(n, dtype=t, device="cuda")
    slot, entry = e(100, torch.int32), e(100, torch.int64)
    ws = csa2.workspace(csa2.page_tables_workspace_size(2))

    def step(add):
        csa2.page_tables(2, have, i32(add), P, table, 4, 10, free, n_free, n_free, have, ws, n_rows=100, slot=slot,
                         entry=entry, n_kept=i32(kept))
        assert csa2.check(ws) == (0, 0)

    step([-100, 0])
    assert table[0].tolist()[:2] == [0, 1] and n_free.item() == 5  # nothing of the shared pages came back
    # the caller: a free page in place of the one entry 28 lies in (its 28 entries are copied there), none kept
    own = free[n_free.item() - 1].item()
    n_free -= 1
    table[0, 0] = own
    kept[0] = 0
    step([100, 0])
    assert set(slot.tolist()) == {own, 6} and entry.tolist() == [*range(28, 64), *range(64)]
    step([-128, -200])
    got = free[:n_free.item()].tolist()
    assert sorted(got) == [2, 3, 5, 6, 7, 8, 9] and have.tolist() == [0, 0]  # all but the shared pages 0 and 1


def test_padded_steps_from_a_graph():
    """One captured step of four requests on a shared prompt, for up to 13 new entries: tables, appends of entries
    and window rows through the padded map, the window without dropped tokens, and attention.  A model in Python
    follows the lengths and the window; the reference reads the planes' and the ring's own bytes."""
    rng = np.random.default_rng(33)
    B, P, d, n_pages, max_pages, rows, n_win, prompt = 4, 16, 128, 40, 8, 13, 8, 32
    planes = csa2.Planes.empty(n_pages, P)
    for t in (planes.kv_codes, planes.kv_scales, planes.ix_codes, planes.ix_scales):
        t.zero_()
    lat, ki = (to_dev(rng.standard_normal((2 * P, n)).astype(np.float32)) for n in (512, 128))
    csa2.quantize_entries(planes, lat, ki, 2 * P)  # the prompt: pages 0 and 1, full
    i32 = lambda v: to_dev(np.asarray(v, np.int32))
    table = np.full((B, max_pages), -1, np.int32)
    table[:, :2] = [0, 1]
    table, have, add, kept = i32(table), i32([prompt] * B), i32([0] * B), i32([2] * B)
    free, n_free = i32([*range(2, n_pages), -1, -1]), i32([n_pages - 2])
    e = lambda *n, t=torch.int32: torch.empty(n, dtype=t, device="cuda")
    query, slot, entry, pos = e(rows), e(rows), e(rows, t=torch.int64), e(rows, t=torch.int64)
    w = [to_dev(rng.standard_normal(s).astype(np.float32) * d ** -0.5).to(torch.bfloat16)
         for s in ((d, 512), (d, 512), (512, 128))]
    hidden, latent = e(rows, 1, d, t=torch.bfloat16), e(rows, 512, t=torch.float32)
    ring, ring_pos = e(B, n_win, 512, t=torch.uint8), e(B, n_win, t=torch.int64)
    ring.zero_()
    ring_pos.fill_(-1)
    lo, q, out, lse = torch.zeros_like(ring_pos[:, 0]), e(B, H, D, t=torch.bfloat16), e(B, H, D, t=torch.float32), e(B, H, t=torch.float32)
    wst, wsa = (csa2.workspace(n) for n in (csa2.page_tables_workspace_size(B), csa2.cache_append_workspace_size(rows, d, 1)))
    wsp = csa2.workspace(csa2.prefix_attn_workspace_size(B, 1, prompt, 64, n_win))
    start, shared, pages, win = i32([0, B]), i32([prompt]), csa2.pages(table, n_pages), csa2.window(ring_pos, lo)

    def step():
        csa2.page_tables(B, have, add, P, table, max_pages, n_pages, free, n_free, n_free, have, wst, n_rows=rows,
                         query=query, slot=slot, entry=entry, pos=pos, n_kept=kept)
        csa2.cache_append(hidden, rows, d, *w, 1, planes, n_pages, slot, entry, wsa)
        ring_pos.copy_(torch.where(ring_pos < have[:, None], ring_pos, -1))  # dropped tokens
        csa2.swa_append(latent, rows, pos, B, ring, n_win, query=query, ring_pos=ring_pos)
        csa2.prefix_attn_decode(planes, pages, B, have, 1, start, shared, prompt, 64, ring, n_win, q, SCALE, out, wsp,
                                lse_out=lse, win=win)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    latent.zero_(), hidden.zero_(), q.zero_()
    with torch.cuda.stream(st):
        step()  # no new entry: nothing but padding
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step()
    st.synchronize()
    count, window = [prompt] * B, [dict() for _ in range(B)]
    for new in ([1, 1, 1, 1], [3, 0, 9, 0], [-2, 0, -6, 2], [0, 0, 0, 0], [1, 12, -3, -1], [0, -4, 10, 2], [-1, 3, 0, 9]):
        # random bytes in the padding's rows too
        hidden.copy_(torch.randn(rows, 1, d, generator=torch.Generator().manual_seed(count[1])))
        x = torch.randn(rows, 512, generator=torch.Generator().manual_seed(count[2]))
        q.copy_(torch.randn(B, H, D, generator=torch.Generator().manual_seed(count[3])))
        latent.copy_(x)
        add.copy_(i32(new))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        st.synchronize()
        for ws in (wst, wsa, wsp):
            assert csa2.check(ws) == (0, 0)
        at = 0
        for b in range(B):
            window[b] = {p: v for p, v in window[b].items() if p < count[b] + new[b]}
            for p in range(count[b], count[b] + max(new[b], 0)):
                window[b].pop(p - n_win, None)
                window[b][p] = x[at].to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                at += 1
            count[b] += new[b]
        assert have.tolist() == count and query.tolist()[at:] == [-1] * (rows - at)
        t, codes, scales, rp, swa = (v.cpu().numpy() for v in (table, planes.kv_codes, planes.kv_scales, ring_pos, ring))
        ref = []
        for b in range(B):
            seen = {int(rp[b, i]): swa[b, i] for i in range(n_win) if rp[b, i] >= 0}
            assert seen.keys() == window[b].keys() and all(np.array_equal(seen[p], window[b][p]) for p in seen)
            j = np.arange(count[b])
            r = t[b, j // P].astype(np.int64) * P + j % P
            assert len(set(r)) == count[b] and (scales[r] != 0).any(1).all()
            x_b = np.concatenate([decode(codes[r], scales[r]), F8[np.stack(list(seen.values()))] if seen else np.zeros((0, D))])
            ref.append(attention(x_b, q[b].double().cpu().numpy(), SCALE))
        o, l, bound, lb = (np.stack(z) for z in zip(*ref))
        assert (np.abs(out.double().cpu().numpy() - o) <= bound + 2.0 ** -22 * np.abs(o)).all()
        assert (np.abs(lse.double().cpu().numpy() - l) <= lb).all()
