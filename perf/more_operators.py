"""Measured cases of the operators that a serving loop with draft trees runs on the paged cache: attention
of a tree of drafted tokens, the commit of the accepted path, appending latents with the rotation on
the way, and rotary positions by themselves.

Each operator has a plain form (elementary torch operations in 32 bits, in 64 where angles or the codec's
borders want it, rounded once at the end) and the framework's own calls.  A cache is a pool of pages of
`page` entries: 512 E2M1 codes with one E4M3 scale per 16 (main), 128 E2M1 codes with one E8M0 scale per
32 (indexer key).  Attention returns bf16 outputs [B][64][512] and the fp32 logsumexp [B][64].  Planes are
returned as they are held, two codes to a byte: the codec's bytes are decided by its definition, so equal
bytes are asked for, and reading them back as values would cost more than the append.
"""
import math
import random

import numpy as np
import torch

own = False

H, D, KEY, WIN = 64, 512, 128, 128
SCALE = 1.0 / math.sqrt(D)
ROPE_BASE, EPS = 10000.0, 1e-6
YARN, ORIGINAL, BETA_FAST, BETA_SLOW = 16.0, 65536, 32.0, 1.0  # contexts of 2^20 tokens from 2^16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------ cases

def _tree(name, R, tokens, n, page, entries, window, extras, ragged, lens):
    return {"name": name, "op": "tree", "R": R, "tokens": tokens, "n": n, "page": page, "entries": entries,
            "window": window, "extras": extras, "ragged": ragged, "lens": lens}


def _commit(name, R, tokens, n, page, ragged, lens):
    return {"name": name, "op": "commit", "R": R, "tokens": tokens, "n": n, "page": page, "ragged": ragged, "lens": lens}


def _append(name, rows, page, bf16, norm, scaled, pad, lens):
    return {"name": name, "op": "append", "rows": rows, "page": page, "bf16": bf16, "norm": norm, "scaled": scaled,
            "pad": pad, "lens": lens}


def _rope(name, rows, heads, dim, first, n_rot, halves, bf16, scaled, inverse, gap, lens):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "dim": dim, "first": first, "n_rot": n_rot,
            "halves": halves, "bf16": bf16, "scaled": scaled, "inverse": inverse, "gap": gap, "lens": lens}


def listed():
    return [
        # one request that verifies eight drafted tokens at a 4,096-entry context: the latency of a step
        _tree("tree 1 x 8 on 4096", 1, 8, 4096, 64, True, True, False, False, 1),
        # batch 16 at a 1,048,576-token context compressed 128 times (drafts have no entries yet, window rows
        # alone), query norm, scaled rotation and sink on
        _tree("tree 16 x 16 on 8192", 16, 16, 8192, 64, False, True, True, False, 2),
        # a mixed serving batch: trees of 0 to 32 tokens, ragged contexts in small pages, padded queries
        _tree("tree ragged 48 x 32 on 4001", 48, 32, 4001, 16, True, True, False, True, 3),
        # full trees on long contexts: the largest call
        _tree("tree 4 x 64 on 65000", 4, 64, 65000, 128, True, False, True, False, 4),
        # after that step: the accepted tokens of 16 requests move up, their window rows enter the ring
        _commit("commit 16 x 16", 16, 16, 512, 64, False, 5),
        # a large batch of full trees, ragged
        _commit("commit ragged 256 x 64", 256, 64, 500, 16, True, 6),
        # one decode step of a batch of 128: a latent and an indexer key each, norm and scaled rotation
        _append("append decode 128", 128, 64, False, True, True, 3, 7),
        # 131,072 tokens compressed four times enter the cache in one prefill chunk
        _append("append prefill 32768", 32768, 64, False, True, True, 0, 8),
        # indexer queries of a decode step: 32 heads of 128 channels, half of them rotated, halves layout
        _rope("rope decode 128 x 32", 128, 32, 128, 64, 64, True, True, True, False, 0, 9),
        # the same of a long prefill, cut out of a fused projection: the largest
        _rope("rope prefill 32768 x 32", 32768, 32, 128, 0, 64, True, True, True, False, 512, 10),
        # the gradient of the latents' rotation (interleaved, last 64 of 512 channels), odd rows, fp32
        _rope("rope gradient 16385 x 512", 16385, 1, 512, 448, 64, False, False, False, True, 0, 11),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    lens = rng.randrange(1 << 20)
    op = rng.choice(("tree", "tree", "tree", "commit", "append", "rope", "rope"))
    page = rng.choice((8, 16, 24, 32, 64, 100, 128, 256))
    if op == "tree":
        tokens = _log_int(rng, 1, 64)
        R = _log_int(rng, 1, 64)
        n = _log_int(rng, 1, min(65000, max(1, (4 * 64 * 65000) // (R * tokens * 2))))
        c = _tree("", R, tokens, n, page, rng.random() < 0.6, rng.random() < 0.7, rng.random() < 0.5,
                  rng.random() < 0.6, lens)
    elif op == "commit":
        c = _commit("", _log_int(rng, 1, 256), _log_int(rng, 1, 64), _log_int(rng, 1, 512), page, rng.random() < 0.6, lens)
    elif op == "append":
        c = _append("", _log_int(rng, 1, 32768), page, rng.random() < 0.4, rng.random() < 0.7, rng.random() < 0.6,
                    rng.randrange(8), lens)
    else:
        dim = rng.choice((64, 96, 128, 192, 256, 512))
        heads = rng.choice((1, 2, 8, 32, 64, 5))
        n_rot = rng.choice((32, 64, dim, dim // 2))
        c = _rope("", _log_int(rng, 1, min(32768, (1 << 26) // (heads * dim))), heads, dim,
                  rng.choice((0, dim - n_rot)), n_rot, rng.random() < 0.5, rng.random() < 0.6, rng.random() < 0.5,
                  rng.random() < 0.4, rng.choice((0, 0, 64, 7)), lens)
    del c["name"]
    return c


def _pages_of(n, page):
    return -(-n // page)


def _tree_lens(c):
    """Per request: entries of its context, tokens, their parents, the first token's position, ring rows filled;
    and queries behind the last tree."""
    r = random.Random(c["lens"])
    n, parents, rows = [], [], []
    for g in range(c["R"]):
        T, have = c["tokens"], c["n"]
        if c["ragged"] and g > 0:
            T = r.choice((r.randint(0, T), r.randint(0, T), _log_int(r, 1, T)))
            have = r.choice((r.randint(0, have), _log_int(r, 1, have)))
            if g == 2:
                T, have = max(T, 1), 0  # a request that begins
        # a few roots, then mostly children of recent tokens
        parents.append([-1 if t == 0 or r.random() < 0.1 else r.randint(max(0, t - 6), t - 1) for t in range(T)])
        n.append(have)
        rows.append(WIN if not c["ragged"] or r.random() < 0.7 else r.randint(0, WIN))
    pos0 = [max(h, w) if not c.get("extras") else r.randint(1 << 19, (1 << 20) - 1) for h, w in zip(n, rows)]
    return n, parents, pos0, rows, 2 if c["ragged"] else 0


def _ancestors(parents):
    """Per token, itself and its ancestors, from the root on."""
    chain = []
    for t, p in enumerate(parents):
        chain.append((chain[p] if p >= 0 else []) + [t])
    return chain


def _commit_lens(c):
    """Per request: entries of its context, tokens, the accepted path."""
    r = random.Random(c["lens"])
    n, tokens, paths = [], [], []
    for g in range(c["R"]):
        T, have = c["tokens"], c["n"]
        if c["ragged"] and g > 0:
            T, have = r.randint(0, T), r.randint(0, have)
        size = r.randint(0, T) if c["ragged"] else min(T, 1 + T // 3)
        paths.append(sorted(r.sample(range(T), size)))
        n.append(have)
        tokens.append(T)
    return n, tokens, paths


def work(case):
    c = case
    if c["op"] == "tree":
        n, parents, _, rows, pad = _tree_lens(c)
        pairs = reads = 0
        B = pad
        for have, par, w in zip(n, parents, rows):
            T = len(par)
            own_rows = sum(len(a) for a in _ancestors(par))
            pairs += T * have + own_rows * c["entries"]
            if T:
                reads += (have + T * c["entries"]) * 288 + _pages_of(have + T * c["entries"], c["page"]) * 4
            if c["window"] and T:
                pairs += T * w + own_rows  # the ring rows that depth takes out of a window are few
                reads += w * D + WIN * 8 + T * D
            B += T
        return {"bytes": reads + B * (2 * H * D * 2 + H * 4 + 4 + 8) + c["R"] * 8, "flops": pairs * H * D * 4}
    if c["op"] == "commit":
        _, tokens, paths = _commit_lens(c)
        moved = sum(i != a for p in paths for i, a in enumerate(p))
        kept = sum(len(p) for p in paths)
        # entries that change place, window rows with their positions, paths; lengths in and out
        return {"bytes": moved * 2 * 356 + kept * (2 * D + 8 + 4) + c["R"] * 28, "flops": 0}
    if c["op"] == "append":
        size = 2 if c["bf16"] else 4
        return {"bytes": c["rows"] * ((D + KEY) * size + 356 + 20) + D * 4 * c["norm"], "flops": c["rows"] * D * 6}
    size = 2 if c["bf16"] else 4
    return {"bytes": c["rows"] * (c["heads"] * c["dim"] * size * 2 + 8), "flops": c["rows"] * c["heads"] * c["n_rot"] * 3}


# ----------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


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


def _tables(n, page, seed, spare):
    """Page tables of requests of n[g] entries, pages in random order."""
    count = sum(_pages_of(x, page) for x in n) + spare
    ids = np.random.RandomState(seed % (1 << 32)).permutation(count).astype(np.int32)
    table = np.full((len(n), max(1, max(_pages_of(x, page) for x in n))), -1, np.int32)
    at = 0
    for g, x in enumerate(n):
        k = _pages_of(x, page)
        table[g, :k] = ids[at:at + k]
        at += k
    return torch.from_numpy(table).cuda(), count, ids


def _window(R, n_rows, pos0, gen):
    """Rings [R][WIN][512] e4m3 whose last n_rows[g] positions before pos0[g] are filled, and the positions."""
    ring = torch.randn((R, WIN, D), device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8)
    at = np.full((R, WIN), -1, np.int64)
    for g in range(R):
        p = np.arange(pos0[g] - n_rows[g], pos0[g])
        at[g, p % WIN] = p
    return ring, torch.from_numpy(at).cuda()


def _prepare_tree(c, seed):
    n, parents, pos0, rows, pad = _tree_lens(c)
    R, P, gen = c["R"], c["page"], _gen(seed)
    T = [len(p) for p in parents]
    B = sum(T) + pad
    total = [h + t * c["entries"] for h, t in zip(n, T)]
    table, n_pages, _ = _tables(total, P, seed, 3)
    codes, scales = _quantized(n_pages * P, gen)
    start = np.concatenate([[0], np.cumsum(T)]).tolist()
    depth = [len(a) - 1 for par in parents for a in _ancestors(par)]
    s = {"c": c, "R": R, "B": max(B, 1), "P": P, "n_pages": n_pages, "codes": codes, "scales": scales, "table": table,
         "n": _i32(n), "n_max": max(n), "start": _i32(start), "most": max(1, max(T)),
         "parent": _i32([p for par in parents for p in par] + [-1] * (max(B, 1) - sum(T))),
         "q_pos": _i64([pos0[g] + d for g, d in zip(np.repeat(np.arange(R), T), depth)] + [0] * (max(B, 1) - sum(T))),
         "q": torch.randn((max(B, 1), H, D), device="cuda", generator=gen).to(torch.bfloat16),
         "ring": None, "ring_pos": None, "draft": None, "norm": None, "sink": None}
    if c["window"]:
        s["ring"], s["ring_pos"] = _window(R, rows, pos0, gen)
        s["draft"] = torch.randn((s["B"], D), device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8)
    if c["extras"]:
        s["norm"] = 1.0 + 0.3 * torch.randn(D, device="cuda", generator=gen)
        s["sink"] = 2.0 * torch.randn(H, device="cuda", generator=gen)
    if own:  # what a serving loop allocates once: the planes' handle, the outputs and the workspace
        import compressed_sparse_attention_nvfp4_gb300 as csa2

        e = lambda *k: torch.empty(k, dtype=torch.uint8, device="cuda")  # noqa: E731
        s["planes"] = csa2.Planes(codes, scales, e(n_pages * P, 64), e(n_pages * P, 4), P)
        s["pages"] = csa2.pages(table, n_pages)
        s["trees"] = csa2.trees(s["start"], s["parent"], R, s["B"], s["most"], entries=c["entries"])
        s["nr"] = csa2.norm_rope(s["norm"], EPS, True, ROPE_BASE) if c["extras"] else None
        s["scaling"] = csa2.rope_scaling(csa2.SCALE_YARN, YARN, ORIGINAL, BETA_FAST, BETA_SLOW) if c["extras"] else None
        s["out"] = torch.empty((s["B"], H, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((s["B"], H), dtype=torch.float32, device="cuda")
        s["ws"] = csa2.workspace(csa2.tree_attn_workspace_size(R, s["B"], s["most"], s["n_max"],
                                                               WIN if c["window"] else 0))
    return s


def _prepare_commit(c, seed):
    n, T, paths = _commit_lens(c)
    R, P, gen = c["R"], c["page"], _gen(seed)
    table, n_pages, _ = _tables([h + t for h, t in zip(n, T)], P, seed, 3)
    N = n_pages * P + 1
    codes, scales = _quantized(N, gen)
    u8 = lambda *k: torch.randint(0, 256, k, dtype=torch.uint8, device="cuda", generator=gen)  # noqa: E731
    path = np.full((R, c["tokens"]), -1, np.int32)
    for g, p in enumerate(paths):
        path[g, :len(p)] = p
    B = max(1, sum(T))
    ring, ring_pos = _window(R, [min(WIN, h) for h in n], n, gen)
    s = {"c": c, "R": R, "P": P, "codes": codes, "scales": scales, "ix_codes": u8(N, 64), "ix_scales": u8(N, 4),
         "table": table, "n": _i32(n), "start": _i32(np.concatenate([[0], np.cumsum(T)]).tolist()),
         "accept": _i32([len(p) for p in paths]), "path": torch.from_numpy(path).cuda(), "pos0": _i64(n),
         "draft": torch.randn((B, D), device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8),
         "ring": ring, "ring_pos": ring_pos}
    if own:
        import compressed_sparse_attention_nvfp4_gb300 as csa2

        s["planes"] = csa2.Planes(codes, scales, s["ix_codes"], s["ix_scales"], P)
        s["pages"] = csa2.pages(table, n_pages)
        s["trees"] = csa2.trees(s["start"], None, R, B, c["tokens"], entries=True)
        s["new"] = torch.empty(R, dtype=torch.int32, device="cuda")
        s["ws"] = csa2.workspace(csa2.tree_commit_workspace_size(R))
    return s


def _prepare_append(c, seed):
    rows, P, gen = c["rows"], c["page"], _gen(seed)
    table, n_pages, ids = _tables([rows], P, seed, 3)
    dtype = torch.bfloat16 if c["bf16"] else torch.float32
    e = np.arange(rows)
    slot, entry = ids[e // P].astype(np.int32), (e % P).astype(np.int64)
    pos = np.random.RandomState(seed % (1 << 32)).randint(0, 1 << 20, rows).astype(np.int64)
    # the padding rows of a fixed-size step lie behind
    slot, entry, pos = (np.concatenate([a, np.full(c["pad"], -1, a.dtype)]) for a in (slot, entry, pos))
    R, N = rows + c["pad"], n_pages * P + 1
    z = lambda *k: torch.zeros(k, dtype=torch.uint8, device="cuda")  # noqa: E731
    s = {"c": c, "R": R, "P": P, "n_pages": n_pages,
         "x": torch.randn((R, D), device="cuda", generator=gen).to(dtype),
         "key": torch.randn((R, KEY), device="cuda", generator=gen).to(dtype),
         "norm": 1.0 + 0.3 * torch.randn(D, device="cuda", generator=gen) if c["norm"] else None,
         "slot": torch.from_numpy(slot).cuda(), "entry": torch.from_numpy(entry).cuda(), "pos": torch.from_numpy(pos).cuda(),
         "codes": z(N, 256), "scales": z(N, 32), "ix_codes": z(N, 64), "ix_scales": z(N, 4)}
    if own:
        import compressed_sparse_attention_nvfp4_gb300 as csa2

        s["planes"] = csa2.Planes(s["codes"], s["scales"], s["ix_codes"], s["ix_scales"], P)
        s["nr"] = csa2.norm_rope(s["norm"], EPS, True, ROPE_BASE)
        s["scaling"] = csa2.rope_scaling(csa2.SCALE_YARN, YARN, ORIGINAL, BETA_FAST, BETA_SLOW) if c["scaled"] else None
        s["rot"] = csa2.rotary(64, 64, csa2.ROPE_HALVES, ROPE_BASE, scaling=s["scaling"])
        s["ws"] = csa2.workspace(csa2.latent_append_workspace_size(R))
    return s


def _prepare_rope(c, seed):
    gen = _gen(seed)
    dtype = torch.bfloat16 if c["bf16"] else torch.float32
    wide = c["heads"] * c["dim"] + c["gap"]  # the heads lie in front of a fused projection's other channels
    x = torch.randn((c["rows"], wide), device="cuda", generator=gen).to(dtype)
    s = {"c": c, "x": x[:, :c["heads"] * c["dim"]].view(c["rows"], c["heads"], c["dim"]),
         "pos": torch.randint(0, 1 << 20, (c["rows"],), device="cuda", generator=gen)}
    if own:
        import compressed_sparse_attention_nvfp4_gb300 as csa2

        scaling = csa2.rope_scaling(csa2.SCALE_YARN, YARN, ORIGINAL, BETA_FAST, BETA_SLOW) if c["scaled"] else None
        s["rot"] = csa2.rotary(c["n_rot"], c["first"], csa2.ROPE_HALVES if c["halves"] else csa2.ROPE_INTERLEAVED,
                               ROPE_BASE, scaling=scaling)
        s["out"] = torch.empty((c["rows"], c["heads"], c["dim"]), dtype=dtype, device="cuda")
    return s


def prepare(case, seed):
    return {"tree": _prepare_tree, "commit": _prepare_commit, "append": _prepare_append,
            "rope": _prepare_rope}[case["op"]](case, seed)


# ------------------------------------------------------------------------------------ plain forms

def _theta(n_rot, scaled):
    """Turn of each pair a position, fp64; YaRN: pairs that turn often as they are, rare ones slowed down."""
    i = torch.arange(n_rot // 2, device="cuda", dtype=torch.float64)
    theta = ROPE_BASE ** (-2.0 * i / n_rot)
    if not scaled:
        return theta
    at = lambda turns: n_rot * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(ROPE_BASE))  # noqa: E731
    low, high = max(math.floor(at(BETA_FAST)), 0), min(math.ceil(at(BETA_SLOW)), n_rot - 1)
    ramp = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
    return theta * (1.0 - ramp) + theta / YARN * ramp


def _turned(x, pos, first, n_rot, halves, scaled, inverse):
    """x [..., dim] with its pairs turned by pos (whose shape broadcasts against x's without the channels)."""
    angle = pos.double()[..., None] * _theta(n_rot, scaled)
    cos, sin = angle.cos().to(x.dtype), angle.sin().to(x.dtype)
    if inverse:
        sin = -sin
    r = x[..., first:first + n_rot]
    a, b = (r[..., :n_rot // 2], r[..., n_rot // 2:]) if halves else (r[..., 0::2], r[..., 1::2])
    u, v = a * cos - b * sin, a * sin + b * cos
    r = torch.cat([u, v], -1) if halves else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([x[..., :first], r, x[..., first + n_rot:]], -1)


def _decoded(codes, scales):
    """fp32 values of cache entries: E2M1 codes (low nibble first) times the E4M3 scale of their 16 channels."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    byte = torch.arange(256, device="cuda")
    pair = torch.stack([lut[byte % 16], lut[byte // 16]], -1)
    x = pair[codes.int()].view(-1, D // 16, 16)
    return (x * scales.view(torch.float8_e4m3fn).float()[..., None]).view(-1, D)


def _plain_tree(s):
    c, R, B, P, T = s["c"], s["R"], s["B"], s["P"], s["most"]
    q = s["q"].float()
    if s["norm"] is not None:
        q = s["norm"] * (q / torch.sqrt(q.square().mean(-1, keepdim=True) + EPS))
        q = _turned(q, s["q_pos"][:, None], 448, 64, False, True, False)
    # requests side by side, padded to the largest tree
    t = torch.arange(T, device="cuda")
    first, size = s["start"][:-1].long()[:, None], (s["start"][1:] - s["start"][:-1]).long()[:, None]
    live = t < size
    at = torch.where(live, first + t, 0)
    parent = torch.where(live, s["parent"][at].long(), -1)
    step = (parent[..., None] == t).float() + torch.eye(T, device="cuda")
    kin = (torch.linalg.matrix_power(step, 64) > 0) & live[..., None]  # [R][token][ancestor or itself]
    depth = kin.sum(-1) - 1
    n = s["n"].long()[:, None]
    L = s["n_max"] + (T if c["entries"] else 0)
    j = torch.arange(L, device="cuda")[None]
    row = s["table"].long()[:, (j[0] // P).clamp(max=s["table"].shape[1] - 1)] * P + j % P
    there = j < n + (size if c["entries"] else 0)
    x = _decoded(s["codes"], s["scales"])[torch.where(there, row, 0)]
    kin_at = torch.gather(kin, 2, (j - n).clamp(0, T - 1)[:, None].expand(R, T, L))
    seen = (j < n)[:, None] | (kin_at & (there & (j >= n))[:, None])
    if s["ring"] is not None:
        f8 = lambda v: v.view(torch.float8_e4m3fn).float()  # noqa: E731
        x = torch.cat([x, f8(s["ring"]), f8(s["draft"])[at]], 1)
        p = s["q_pos"][at]
        ring = (s["ring_pos"][:, None] >= (p - WIN + 1).clamp(min=0)[..., None]) & (
            s["ring_pos"][:, None] < (p - depth)[..., None])
        seen = torch.cat([seen, ring, kin & (depth[..., None] - depth[:, None] < WIN)], 2)
    z = torch.matmul(q[at].view(R, T * H, D), x.transpose(1, 2)).view(R, T, H, -1) * SCALE
    z = torch.where(seen[:, :, None], z, -math.inf)
    top = z.amax(-1, keepdim=True) if z.shape[-1] else torch.full((R, T, H, 1), -math.inf, device="cuda")
    sink = s["sink"][:, None] if s["sink"] is not None else torch.full((H, 1), -math.inf, device="cuda")
    top = torch.maximum(top, sink)
    ref = torch.where(top == -math.inf, 0.0, top)
    prob = torch.exp(z - ref)
    den = prob.sum(-1, keepdim=True) + torch.exp(sink - ref)
    o = torch.matmul(prob.view(R, T * H, -1), x).view(R, T, H, D)
    o = torch.where(den > 0, o / den, 0.0)
    # back to queries; those behind the last tree see nothing
    b = torch.arange(B, device="cuda")
    g = torch.searchsorted(s["start"].long(), b, right=True) - 1
    some, g = (g < R)[:, None, None], g.clamp(max=R - 1)
    k = (b - first[g, 0]).clamp(0, T - 1)
    out = torch.where(some, o[g, k], 0.0)
    if s["norm"] is not None:
        out = _turned(out, s["q_pos"][:, None], 448, 64, False, True, True)
    lse = torch.where(some[..., 0], (ref + torch.log(den))[g, k, :, 0], sink[None, :, 0])
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _plain_commit(s):
    P, R = s["P"], s["R"]
    i = torch.arange(s["path"].shape[1], device="cuda")[None]
    kept = i < s["accept"][:, None]
    n, g = s["n"].long()[:, None], torch.arange(R, device="cuda")[:, None]
    # what is not accepted moves from the row behind the pages to itself
    row = lambda e: torch.where(kept, s["table"].long()[g, e // P] * P + e % P, s["codes"].shape[0] - 1)  # noqa: E731
    src = row(torch.where(kept, n + s["path"], 0)).flatten()
    dst = row(torch.where(kept, n + i, 0)).flatten()
    planes = (s["codes"], s["scales"], s["ix_codes"], s["ix_scales"])
    moved = torch.cat([p[src] for p in planes], 1)
    s["codes"][dst], s["scales"][dst] = moved[:, :256], moved[:, 256:288]
    s["ix_codes"][dst], s["ix_scales"][dst] = moved[:, 288:352], moved[:, 352:]
    # window rows: place w takes the accepted token i with (pos0 + i) % WIN = w
    w = torch.arange(WIN, device="cuda")[None]
    take = (w - s["pos0"][:, None]) % WIN
    hit = take < s["accept"][:, None]
    take = take.clamp(max=s["path"].shape[1] - 1)
    from_row = (s["start"][:-1].long()[:, None] + s["path"].long().gather(1, take)).clamp(0, s["draft"].shape[0] - 1)
    s["ring"].copy_(torch.where(hit[..., None], s["draft"][from_row], s["ring"]))
    s["ring_pos"].copy_(torch.where(hit, s["pos0"][:, None] + take, s["ring_pos"]))
    new = s["accept"] - (s["start"][1:] - s["start"][:-1])
    return _commit_outputs(s, new)


def _commit_outputs(s, new):
    return {"codes": s["codes"], "scales": s["scales"], "ix_codes": s["ix_codes"], "ix_scales": s["ix_scales"],
            "ring": s["ring"].view(torch.float8_e4m3fn), "ring_pos": s["ring_pos"], "new": new}


def _e2m1(v):
    """Codes of the nearest E2M1 value (ties to the even code, saturating); a negative that rounds to zero keeps its sign."""
    a = v.abs()
    k = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4)).clamp(max=7)
    return k.to(torch.uint8) | torch.signbit(v).to(torch.uint8) * 8


def _packed(code):
    code = code.view(code.shape[0], -1, 2)
    return code[..., 0] | code[..., 1] * 16


def _plain_append(s):
    c, R = s["c"], s["R"]
    y, k = s["x"].double(), s["key"].double()
    if s["norm"] is not None:
        y = s["norm"].double() * y / torch.sqrt(y.square().mean(-1, keepdim=True) + float(np.float32(EPS)))
    y = _turned(y, s["pos"], 448, 64, False, c["scaled"], False).float()
    k = _turned(k, s["pos"], 64, 64, True, c["scaled"], False).float()
    g = y.view(R, 32, 16)
    scale = (g.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    f = scale.float()[..., None]
    code = torch.where(f > 0, _e2m1(g / torch.where(f > 0, f, 1.0)), 0)
    h = k.view(R, 4, 32)
    top = h.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)  # floor(log2 top) - 2
    key = torch.where(top > 0, _e2m1((h.double() * torch.exp2(-e.double())).float()), 0)
    # the row behind the pages takes the padding
    row = torch.where(s["slot"] >= 0, s["slot"].long() * s["P"] + s["entry"], s["codes"].shape[0] - 1)
    planes = (s["codes"], s["scales"], s["ix_codes"], s["ix_scales"])
    values = (_packed(code), scale.view(torch.uint8), _packed(key), (e + 127).to(torch.uint8).view(R, 4))
    pad = (s["slot"] < 0)[:, None]
    put = lambda p, v: p.index_copy_(0, row, torch.where(pad, p[row], v))  # noqa: E731
    put(planes[0], values[0]), put(planes[1], values[1]), put(planes[2], values[2]), put(planes[3], values[3])
    return dict(zip(("codes", "scales", "ix_codes", "ix_scales"), planes))


def _plain_rope(s):
    c = s["c"]
    y = _turned(s["x"].float(), s["pos"][:, None], c["first"], c["n_rot"], c["halves"], c["scaled"], c["inverse"])
    return {"out": y.to(s["x"].dtype)}


def run(state):
    s, c = state, state["c"]
    if not own:
        return {"tree": _plain_tree, "commit": _plain_commit, "append": _plain_append, "rope": _plain_rope}[c["op"]](s)
    import compressed_sparse_attention_nvfp4_gb300 as csa2

    if c["op"] == "tree":
        csa2.tree_attn_decode(s["planes"], s["pages"], s["trees"], s["n"], s["n_max"], s["ring"], s["ring_pos"], s["draft"],
                              WIN if s["ring"] is not None else 0, s["q"], s["q_pos"], SCALE, s["out"], s["ws"],
                              lse_out=s["lse"], q_nr=s["nr"], scaling=s["scaling"], sink=s["sink"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "commit":
        csa2.tree_commit(s["planes"], s["pages"], s["trees"], s["n"], s["accept"], s["path"], c["tokens"], s["new"],
                         s["ws"], draft=s["draft"], pos=s["pos0"], ring=s["ring"], ring_pos=s["ring_pos"], n_win=WIN)
        return _commit_outputs(s, s["new"])
    if c["op"] == "append":
        csa2.latent_append(s["x"], s["R"], s["planes"], s["n_pages"], s["slot"], s["entry"], s["ws"], key=s["key"],
                           kv_nr=s["nr"], scaling=s["scaling"], pos=s["pos"], key_rot=s["rot"])
        return {"codes": s["codes"], "scales": s["scales"], "ix_codes": s["ix_codes"], "ix_scales": s["ix_scales"]}
    csa2.rope(s["x"], c["rows"], c["heads"], c["dim"], s["pos"], s["rot"], s["out"], inverse=c["inverse"])
    return {"out": s["out"]}


# --------------------------------------------------------------------------------------- 64 bits

def _spin(pos, n_rot, scaled):
    """exp(i angle) [len(pos)][n_rot / 2], complex128."""
    theta = []
    for i in range(n_rot // 2):
        t = ROPE_BASE ** (-2 * i / n_rot)
        if scaled:
            lo, hi = (n_rot / 2 * math.log(ORIGINAL / (b * 2 * math.pi), ROPE_BASE) for b in (BETA_FAST, BETA_SLOW))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), n_rot - 1)
            slow = min(max((i - lo) / (hi - lo if hi != lo else 1e-3), 0.0), 1.0)
            t = slow * (t / YARN) + (1 - slow) * t
        theta.append(t)
    a = pos.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device="cuda")
    return torch.polar(torch.ones_like(a), a)


def _exact_tree(c, seed):
    s = _prepare_tree(c, seed)
    n, parents, pos0, _, _ = _tree_lens(c)
    f8 = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    f4 = torch.tensor([(-1) ** (v >> 3) * E2M1[v & 7] for v in range(16)], dtype=torch.float64, device="cuda")
    out = torch.zeros((s["B"], H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((s["B"], H), -math.inf, dtype=torch.float64, device="cuda")
    if s["sink"] is not None:
        lse[:] = s["sink"].double()
    b = 0
    for g, par in enumerate(parents):
        T, chains = len(par), _ancestors(par)
        if not T:
            continue
        total = n[g] + T * c["entries"]
        pages = s["table"][g, :_pages_of(total, s["P"])].long()
        at = (pages[:, None] * s["P"] + torch.arange(s["P"], device="cuda")).flatten()[:total]
        code = s["codes"][at].long()
        x = torch.empty((total, D), dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = f4[code & 15], f4[code >> 4]
        x *= f8[s["scales"][at].long()].repeat_interleave(16, 1)
        kin = torch.zeros((T, T), dtype=torch.bool)
        for t, a in enumerate(chains):
            kin[t, a] = True
        kin = kin.cuda()
        ok = torch.ones((T, n[g]), dtype=torch.bool, device="cuda")
        if c["entries"]:
            ok = torch.cat([ok, kin], 1)
        if s["ring"] is not None:
            x = torch.cat([x, f8[s["ring"][g].long()], f8[s["draft"][b:b + T].long()]])
            p = s["q_pos"][b:b + T, None]
            ring = (s["ring_pos"][g] >= 0) & (s["ring_pos"][g] < pos0[g]) & (s["ring_pos"][g] > p - WIN)
            ok = torch.cat([ok, ring, kin], 1)
        q = s["q"][b:b + T].double()
        turn = None
        if s["norm"] is not None:
            q = s["norm"].double() * q / (q.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
            turn = _spin(s["q_pos"][b:b + T], 64, True)[:, None]
            q[..., 448:] = torch.view_as_real(torch.view_as_complex(q[..., 448:].reshape(T, H, 32, 2)) * turn).flatten(2)
        for t in range(0, T, 16):  # 16 tokens at a time
            m = min(16, T - t)
            z = (SCALE * (q[t:t + m].reshape(m * H, D) @ x.T)).view(m, H, -1)
            z = z.masked_fill(~ok[t:t + m, None], -math.inf)
            if s["sink"] is not None:
                z = torch.cat([z, s["sink"].double().view(1, H, 1).expand(m, H, 1)], 2)
            norm = torch.logsumexp(z, 2)
            w = torch.exp(z - norm[..., None])[..., :x.shape[0]]
            out[b + t:b + t + m] = (w.reshape(m * H, -1) @ x).view(m, H, D)
            lse[b + t:b + t + m] = norm
        if turn is not None:
            o = out[b:b + T]
            o[..., 448:] = torch.view_as_real(torch.view_as_complex(o[..., 448:].reshape(T, H, 32, 2)) * turn.conj()).flatten(2)
        b += T
    return {"out": out, "lse": lse}


def _exact_rope(c, seed):
    s = _prepare_rope(c, seed)
    y = s["x"].double()
    spin = _spin(s["pos"], c["n_rot"], c["scaled"])[:, None]
    if c["inverse"]:
        spin = spin.conj()
    f, h = c["first"], c["n_rot"] // 2
    a, b = (slice(f, f + h), slice(f + h, f + 2 * h)) if c["halves"] else (slice(f, f + 2 * h, 2), slice(f + 1, f + 2 * h, 2))
    turned = torch.complex(y[..., a], y[..., b]) * spin
    y[..., a], y[..., b] = turned.real, turned.imag
    return {"out": y}


def exact(case, seed):
    """Attention's and rotation's outputs from the definition, in 64 bits; bytes and whole numbers have none."""
    if case["op"] == "tree":
        return _exact_tree(case, seed)
    return _exact_rope(case, seed) if case["op"] == "rope" else None
