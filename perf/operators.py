"""Measured cases of the paged-cache operators: page tables and slot maps built on the GPU, attention
over a paged FP4 cache, and attention for a batch whose queries share long prefixes.

Each operator has a plain form (elementary torch operations in 32 bits, angles in 64, rounded once at
the end) and the framework's own calls.  A cache is a pool of pages of `page` entries, 288 bytes each
(512 E2M1 codes, one E4M3 scale per 16); 64 query heads share the 512-channel entry, which is key and
value.  Attention returns bf16 outputs [B][64][512] and the fp32 logsumexp [B][64].
"""
import math
import random

import numpy as np
import torch

own = False

H, D, WIN = 64, 512, 128
SCALE = 1.0 / math.sqrt(D)
ROPE_BASE, EPS = 10000.0, 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------ cases

def _tables(name, B, page, have, new, mode, lens):
    return {"name": name, "op": "tables", "B": B, "page": page, "have": have, "new": new, "mode": mode, "lens": lens}


def _paged(name, B, n, page, window, extras, ragged, lens):
    return {"name": name, "op": "paged", "B": B, "n": n, "page": page, "window": window, "extras": extras,
            "ragged": ragged, "lens": lens}


def _prefix(name, B, G, shared, tail, page, window, extras, ragged, lens):
    return {"name": name, "op": "prefix", "B": B, "G": G, "shared": shared, "tail": tail, "page": page,
            "window": window, "extras": extras, "ragged": ragged, "lens": lens}


def listed():
    return [
        # one decode step of a batch of 128: every request appends one entry, few need a new page
        _tables("tables decode 128", 128, 64, 8192, 1, "append", 1),
        # a step of 256 requests that verifies drafts: some grow, some drop the entries of rejected ones
        _tables("tables rollback 256", 256, 16, 2048, 8, "mixed", 2),
        # prefill chunks of 64 requests enter the cache together: ragged, about 130,000 new entries
        _tables("tables prefill 64", 64, 64, 8192, 4096, "append", 3),
        # a single request at a 4,096-entry context: the latency of one token
        _paged("paged single 4096", 1, 4096, 64, True, False, False, 4),
        # batch 32 at a 1,048,576-token context compressed 128 times, query norm, rotation and sink on
        _paged("paged 32 x 8192", 32, 8192, 64, True, True, False, 5),
        # a mixed serving batch of short contexts in small pages, some requests empty, no window
        _paged("paged ragged 128 x 2000", 128, 2000, 16, False, False, True, 6),
        # long ragged contexts up to the longest the dense attention takes
        _paged("paged ragged 48 x 65536", 48, 65536, 128, True, False, True, 7),
        # two requests on one short system prompt: the smallest call
        _prefix("prefix 2 on 512", 2, 1, 512, 16, 64, True, False, False, 8),
        # batch 32 on one document of 1,048,576 tokens compressed 128 times, each with its own turn
        _prefix("prefix 32 on 8192", 32, 1, 8192, 64, 64, True, True, False, 9),
        # a serving batch over several prompts: ragged groups, odd lengths, padded requests at the end
        _prefix("prefix ragged 101 on 4001", 101, 5, 4001, 300, 16, True, False, True, 10),
        # samples drawn in parallel for one long context: the largest call
        _prefix("prefix 64 on 65000", 64, 1, 65000, 256, 128, False, False, False, 11),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    lens = rng.randrange(1 << 20)
    op = rng.choice(("tables", "paged", "paged", "prefix", "prefix", "prefix"))
    page = rng.choice((8, 16, 24, 32, 64, 100, 128, 256))
    if op == "tables":
        mode = rng.choice(("append", "mixed"))
        c = _tables("", _log_int(rng, 1, 512), page, _log_int(rng, 1, 16384), 1, mode, lens)
        c["new"] = rng.choice((1, _log_int(rng, 2, max(2, 65536 // c["B"]))))
    elif op == "paged":
        B = _log_int(rng, 1, 128)
        n = _log_int(rng, 1, min(65536, (1 << 20) // B))
        c = _paged("", B, n, page, rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.6, lens)
    else:
        B = _log_int(rng, 1, 128)
        shared = _log_int(rng, 1, min(65000, (1 << 21) // B))
        c = _prefix("", B, rng.choice((1, 1, _log_int(rng, 1, B))), shared, _log_int(rng, 1, 500), page,
                    rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.6, lens)
    del c["name"]
    return c


def _pages_of(n, page):
    return -(-n // page)


def _table_lens(c):
    """Entries each request has, gets (negative: drops), and leading pages that it shares with others."""
    r = random.Random(c["lens"])
    have, new, kept = [], [], []
    for b in range(c["B"]):
        h = r.randint(c["have"] // 4, c["have"])
        if c["mode"] == "append":
            n = 1 if c["new"] == 1 else r.randint(0, c["new"])
        else:
            n = max(-h, r.randint(-c["new"], c["new"]))
            if r.random() < 0.05:
                n = -h  # the request has ended: all its pages go back
        have.append(h)
        new.append(n)
        kept.append(r.choice((0, 0, 1, 2)))
    return have, new, kept


def _attn_lens(c):
    """Per query: entries and visible window rows; per group: first query and shared entries."""
    r = random.Random(c["lens"])
    B = c["B"]
    pad = 0
    if c["op"] == "paged":
        n = [c["n"]] * B
        if c["ragged"]:
            n = [c["n"] if b == 0 else r.choice((r.randint(0, c["n"]), r.randint(0, c["n"]), _log_int(r, 1, c["n"])))
                 for b in range(B)]
            if B > 4:
                n[2], n[3] = 0, 1
        start, shared = [0, B], [0]
    else:
        pad = min(2, B - 1) if c["ragged"] else 0
        live = B - pad
        G = min(c["G"], live)
        cuts = sorted(r.sample(range(1, live), G - 1)) if c["ragged"] else [live * g // G for g in range(1, G)]
        start = [0] + cuts + [live]
        shared = [c["shared"] if g == 0 or not c["ragged"] else r.randint(c["shared"] // 4, c["shared"])
                  for g in range(G)]
        n = []
        for g in range(G):
            for _ in range(start[g], start[g + 1]):
                n.append(shared[g] + (r.choice((0, r.randint(0, c["tail"]), r.randint(0, c["tail"])))
                                      if c["ragged"] else c["tail"]))
        n += [0] * pad
    rows = [0] * B
    if c["window"]:
        rows = [WIN if not c["ragged"] or r.random() < 0.7 else r.randint(0, WIN) for _ in range(B)]
        rows = [0 if b >= B - pad else v for b, v in enumerate(rows)]
    return n, rows, start, shared


def work(case):
    c = case
    if c["op"] == "tables":
        have, new, kept = _table_lens(c)
        P = c["page"]
        rows = sum(max(x, 0) for x in new)
        moved = sum(abs(_pages_of(h + x, P) - _pages_of(h, P)) for h, x in zip(have, new))
        # lengths in and out, the row starts, 24 bytes a row (query, slot, entry, position), the pages moved
        return {"bytes": c["B"] * 20 + rows * 24 + moved * 8, "flops": 0}
    n, rows, start, shared = _attn_lens(c)
    pairs = sum(n) + sum(rows)
    entries = sum(n)
    pages = sum(_pages_of(x, c["page"]) for x in n)
    if c["op"] == "prefix":  # a group's shared entries, and their pages' ids, are read once
        for g in range(len(shared)):
            more = start[g + 1] - start[g] - 1
            entries -= more * shared[g]
            pages -= more * (shared[g] // c["page"])
    return {"bytes": entries * 288 + sum(rows) * D + pages * 4 + c["B"] * (2 * H * D * 2 + H * 4 + 4),
            "flops": pairs * H * D * 4}


# ----------------------------------------------------------------------------------------- inputs

def _quantized(n, gen):
    """n entries of N(0, 1) latents in the cache's format: codes [n][256], scales [n][32]."""
    codes = torch.empty((n, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, D // 16), dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for i in range(0, n, 1 << 16):
        k = min(1 << 16, n - i)
        x = torch.randn((k, D // 16, 16), device="cuda", generator=gen)
        s = (x.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
        y = x / s.float()[..., None]
        q = torch.bucketize(y.abs(), edges).to(torch.uint8) | (y < 0).to(torch.uint8) * 8
        q = q.view(k, D // 2, 2)
        codes[i:i + k] = q[..., 0] | q[..., 1] * 16
        scales[i:i + k] = s.view(torch.uint8)
    return codes, scales


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def _prepare_tables(c, seed):
    have, new, kept = _table_lens(c)
    B, P = c["B"], c["page"]
    hp = [_pages_of(h, P) for h in have]
    max_pages = max(max(p, _pages_of(h + x, P)) for p, h, x in zip(hp, have, new))
    need = sum(max(0, _pages_of(h + x, P) - p) for p, h, x in zip(hp, have, new))
    n_pages = sum(hp) + need + 64
    ids = np.random.RandomState(seed % (1 << 32)).permutation(n_pages).astype(np.int32)
    table = np.full((B, max_pages), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :hp[b]] = ids[at:at + hp[b]]
        at += hp[b]
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - at] = ids[at:]
    s = {"c": c, "B": B, "P": P, "n_pages": n_pages, "max_pages": max_pages, "n_rows": sum(max(x, 0) for x in new) + 3,
         "have": _i32(have), "new": _i32(new), "kept": _i32(kept), "table": torch.from_numpy(table).cuda(),
         "free": torch.from_numpy(free).cuda(), "n_free": _i32([n_pages - at])}
    if own:  # what a serving loop allocates once: the outputs and the workspace
        import compressed_sparse_attention_nvfp4_gb300 as csa2

        e = lambda n, t: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
        s.update(n_entries=e(B, torch.int32), n_free_out=e(1, torch.int32), row_start=e(B + 1, torch.int32),
                 query=e(s["n_rows"], torch.int32), slot=e(s["n_rows"], torch.int32),
                 entry=e(s["n_rows"], torch.int64), pos=e(s["n_rows"], torch.int64),
                 ws=csa2.workspace(csa2.page_tables_workspace_size(B)))
    return s


def _prepare_attn(c, seed):
    n, rows, start, shared = _attn_lens(c)
    B, P = c["B"], c["page"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    max_pages = max(1, max(_pages_of(x, P) for x in n))
    group = [-1] * B
    for g in range(len(shared)):
        for b in range(start[g], start[g + 1]):
            group[b] = g
    # whole shared pages are the first query's; a page that is shared in part is every query's own copy
    whole = [shared[g] // P if c["op"] == "prefix" and g >= 0 else 0 for g in group]
    first = [start[g] if g >= 0 else b for b, g in enumerate(group)]
    owned = [_pages_of(n[b], P) - (whole[b] if first[b] != b else 0) for b in range(B)]
    n_pages = sum(owned) + 5
    ids = np.random.RandomState(seed % (1 << 32)).permutation(n_pages).astype(np.int32)
    table = np.full((B, max_pages), -1, np.int32)
    at, src, dst = 0, [], []
    for b in range(B):
        skip = _pages_of(n[b], P) - owned[b]
        table[b, :skip] = table[first[b], :skip]
        table[b, skip:skip + owned[b]] = ids[at:at + owned[b]]
        at += owned[b]
        if first[b] != b and c["op"] == "prefix":
            for j in range(shared[group[b]] % P):
                src.append(int(table[first[b], whole[b]]) * P + j)
                dst.append(int(table[b, whole[b]]) * P + j)
    codes, scales = _quantized(n_pages * P, gen)
    if src:
        codes[_i64(dst)], scales[_i64(dst)] = codes[_i64(src)], scales[_i64(src)]
    s = {"c": c, "B": B, "P": P, "n_pages": n_pages, "max_pages": max_pages, "codes": codes, "scales": scales,
         "table": torch.from_numpy(table).cuda(), "n": _i32(n), "n_max": max(n), "swa": None, "pos": None, "lo": None,
         "q": torch.randn((B, H, D), device="cuda", generator=gen).to(torch.bfloat16), "norm": None, "q_pos": None,
         "sink": None}
    if c["window"]:
        s["swa"] = torch.randn((B, WIN, D), device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8)
        if c["ragged"]:  # requests whose window is not full yet
            s["pos"] = _i64([[j if j < v else -1 for j in range(WIN)] for v in rows])
            s["lo"] = _i64([0] * B)
    if c["extras"]:
        s["norm"] = 1.0 + 0.3 * torch.randn(D, device="cuda", generator=gen)
        s["q_pos"] = torch.randint(1 << 19, 1 << 20, (B,), device="cuda", generator=gen)
        s["sink"] = 2.0 * torch.randn(H, device="cuda", generator=gen)
    if own:  # what a serving loop allocates once: the planes' handle, the outputs and the workspace
        import compressed_sparse_attention_nvfp4_gb300 as csa2

        e = lambda *n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        s["planes"] = csa2.Planes(codes, scales, e(n_pages * P, 64), e(n_pages * P, 4), P)
        s["pages"] = csa2.pages(s["table"], n_pages)
        s["nr"] = csa2.norm_rope(s["norm"], EPS, True, ROPE_BASE) if c["extras"] else None
        s["win"] = csa2.window(s["pos"], s["lo"]) if s["pos"] is not None else None
        s["out"] = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, H), dtype=torch.float32, device="cuda")
        n_swa = WIN if c["window"] else 0
        if c["op"] == "paged":
            size = csa2.paged_attn_workspace_size(B, s["n_max"], n_swa)
        else:
            s["start"], s["shared"] = _i32(start), _i32(shared)
            s["G"], s["shared_max"] = len(shared), max(shared)
            s["own_max"] = max([0] + [n[b] - shared[group[b]] for b in range(B) if group[b] >= 0])
            size = csa2.prefix_attn_workspace_size(B, s["G"], s["shared_max"], s["own_max"], n_swa)
        s["ws"] = csa2.workspace(size)
    return s


def prepare(case, seed):
    return _prepare_tables(case, seed) if case["op"] == "tables" else _prepare_attn(case, seed)


# ------------------------------------------------------------------------------------ plain forms

def _plain_tables(s):
    P, B, n_rows = s["P"], s["B"], s["n_rows"]
    have, new = s["have"].long(), s["new"].long()
    total = have + new
    pc, pa = (have + P - 1) // P, (total + P - 1) // P
    need = torch.where(new >= 0, pa - pc, 0)
    keep = torch.maximum(pa, torch.minimum(s["kept"].long(), pc))
    gone = torch.where(new < 0, pc - keep, 0)
    grow = new.clamp(min=0)
    row_end, need_end, gone_end = grow.cumsum(0), need.cumsum(0), gone.cumsum(0)
    n_free = s["n_free"].long()
    # pages given back go on top of the stack of free pages, in order of request and page
    j = torch.arange(s["n_pages"], device="cuda")
    i = j - n_free
    b = torch.searchsorted(gone_end, i.clamp(min=0), right=True).clamp(max=B - 1)
    page = (keep[b] + i - (gone_end - gone)[b]).clamp(0, s["max_pages"] - 1)
    free = torch.where((i >= 0) & (i < gone_end[-1]), s["table"][b, page], s["free"])
    # new pages come from the top, in order of request and page
    top = n_free + gone_end[-1]
    p = torch.arange(s["max_pages"], device="cuda")[None]
    at = top - 1 - ((need_end - need)[:, None] + p - pc[:, None])
    fresh = (p >= pc[:, None]) & (p < pa[:, None]) & (new >= 0)[:, None]
    table = torch.where(fresh, free[at.clamp(0, s["n_pages"] - 1)], s["table"])
    s["free"].copy_(free)
    s["table"].copy_(table)
    # one row of the map for each new entry, -1 behind the last
    r = torch.arange(n_rows, device="cuda")
    b = torch.searchsorted(row_end, r, right=True).clamp(max=B - 1)
    live = r < row_end[-1]
    e = have[b] + r - (row_end - grow)[b]
    slot = table[b, (e // P).clamp(0, s["max_pages"] - 1)]
    return {"table": table, "free": free, "n_free": (top - need_end[-1]).int(), "n_entries": total.int(),
            "row_start": torch.cat([torch.zeros_like(row_end[:1]), row_end]).int(),
            "query": torch.where(live, b, -1).int(), "slot": torch.where(live, slot, -1),
            "entry": torch.where(live, e % P, -1), "pos": torch.where(live, e, -1)}


def _decoded(codes, scales):
    """fp32 values of cache entries: E2M1 codes (low nibble first) times the E4M3 scale of their 16 channels."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    byte = torch.arange(256, device="cuda")
    pair = torch.stack([lut[byte % 16], lut[byte // 16]], -1)
    x = pair[codes.int()].view(-1, D // 16, 16)
    return (x * scales.view(torch.float8_e4m3fn).float()[..., None]).view(-1, D)


def _queries(s):
    """fp32 query heads, normalised and rotated where asked; and the rotation's cosines and sines."""
    q = s["q"].float()
    if s["norm"] is None:
        return q, None, None
    q = s["norm"] * (q / torch.sqrt(q.square().mean(-1, keepdim=True) + EPS))
    i = torch.arange(32, device="cuda", dtype=torch.float64)
    angle = s["q_pos"].double()[:, None] * ROPE_BASE ** (-i / 32)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x, y = q[..., 448::2], q[..., 449::2]
    turned = torch.stack([x * cos - y * sin, x * sin + y * cos], -1).flatten(-2)
    return torch.cat([q[..., :448], turned], -1), cos, sin


def _plain_attn(s):
    B, P = s["B"], s["P"]
    q, cos, sin = _queries(s)
    j = torch.arange(s["n_max"], device="cuda")
    seen = j[None] < s["n"][:, None]
    row = s["table"].long()[:, j // P] * P + j % P
    x = _decoded(s["codes"], s["scales"])[torch.where(seen, row, 0)]
    if s["swa"] is not None:
        x = torch.cat([x, s["swa"].view(torch.float8_e4m3fn).float()], 1)
        rows = s["pos"] >= s["lo"][:, None] if s["pos"] is not None else torch.ones((B, WIN), dtype=torch.bool, device="cuda")
        seen = torch.cat([seen, rows], 1)
    z = torch.matmul(q, x.transpose(1, 2)) * SCALE
    z = torch.where(seen[:, None], z, -math.inf)
    top = z.amax(-1, keepdim=True) if z.shape[-1] else torch.full((B, H, 1), -math.inf, device="cuda")
    if s["sink"] is not None:
        top = torch.maximum(top, s["sink"][None, :, None])
    ref = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(z - ref)
    den = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        den = den + torch.exp(s["sink"][None, :, None] - ref)
    o = torch.where(den > 0, torch.matmul(p, x) / den, 0.0)
    if cos is not None:  # the output's last 64 channels turn back
        a, b = o[..., 448::2], o[..., 449::2]
        o = torch.cat([o[..., :448], torch.stack([a * cos + b * sin, b * cos - a * sin], -1).flatten(-2)], -1)
    return {"out": o.to(torch.bfloat16), "lse": (ref + torch.log(den))[..., 0]}


def run(state):
    s = state
    op = s["c"]["op"]
    if not own:
        return _plain_tables(s) if op == "tables" else _plain_attn(s)
    import compressed_sparse_attention_nvfp4_gb300 as csa2

    if op == "tables":
        csa2.page_tables(s["B"], s["have"], s["new"], s["P"], s["table"], s["max_pages"], s["n_pages"], s["free"],
                         s["n_free"], s["n_free_out"], s["n_entries"], s["ws"], n_rows=s["n_rows"], query=s["query"],
                         slot=s["slot"], entry=s["entry"], pos=s["pos"], row_start=s["row_start"], n_kept=s["kept"])
        return {"table": s["table"], "free": s["free"], "n_free": s["n_free_out"], "n_entries": s["n_entries"],
                "row_start": s["row_start"], "query": s["query"], "slot": s["slot"], "entry": s["entry"],
                "pos": s["pos"]}
    n_swa = WIN if s["swa"] is not None else 0
    more = dict(lse_out=s["lse"], q_nr=s["nr"], q_pos=s["q_pos"], sink=s["sink"], win=s["win"])
    if op == "paged":
        csa2.paged_attn_decode(s["planes"], s["pages"], s["B"], s["n"], s["n_max"], s["swa"], n_swa, s["q"], SCALE,
                               s["out"], s["ws"], **more)
    else:
        csa2.prefix_attn_decode(s["planes"], s["pages"], s["B"], s["n"], s["G"], s["start"], s["shared"],
                                s["shared_max"], s["own_max"], s["swa"], n_swa, s["q"], SCALE, s["out"], s["ws"],
                                **more)
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """out and lse from the definition, in 64 bits, one query at a time; whole numbers need none."""
    if case["op"] == "tables":
        return None
    s = _prepare_attn(case, seed)
    n, rows, _, _ = _attn_lens(case)
    f8 = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    f4 = torch.tensor([(-1) ** (v >> 3) * E2M1[v & 7] for v in range(16)], dtype=torch.float64, device="cuda")
    outs, lses = [], []
    for b in range(case["B"]):
        pages = s["table"][b, :_pages_of(n[b], s["P"])].long()
        at = (pages[:, None] * s["P"] + torch.arange(s["P"], device="cuda")).flatten()[:n[b]]
        code = s["codes"][at].long()
        x = torch.empty((n[b], D), dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = f4[code & 15], f4[code >> 4]
        x *= f8[s["scales"][at].long()].repeat_interleave(16, 1)
        if s["swa"] is not None:
            x = torch.cat([x, f8[s["swa"][b, :rows[b]].long()]])
        q = s["q"][b].double()
        turn = None
        if s["norm"] is not None:
            q = s["norm"].double() * q / (q.pow(2).mean(1, keepdim=True) + EPS).sqrt()
            t = s["q_pos"][b].double() * torch.tensor([ROPE_BASE ** (-i / 32) for i in range(32)],
                                                      dtype=torch.float64, device="cuda")
            turn = torch.polar(torch.ones_like(t), t)
            q[:, 448:] = torch.view_as_real(torch.view_as_complex(q[:, 448:].reshape(H, 32, 2)) * turn).flatten(1)
        z = SCALE * (q @ x.T)
        if s["sink"] is not None:
            z = torch.cat([z, s["sink"].double()[:, None]], 1)
        if z.shape[1] == 0:
            outs.append(torch.zeros((H, D), dtype=torch.float64, device="cuda"))
            lses.append(torch.full((H,), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        lse = torch.logsumexp(z, 1)
        o = torch.exp(z - lse[:, None])[:, :x.shape[0]] @ x
        if turn is not None:
            o[:, 448:] = torch.view_as_real(torch.view_as_complex(o[:, 448:].reshape(H, 32, 2)) * turn.conj()).flatten(1)
        outs.append(o)
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
