"""Plain references of the paged-cache operators: page tables with Python lists, attention in numpy
float64, and the error bound that the kernels' roundings allow."""
from __future__ import annotations

import math

import numpy as np

H, D = 64, 512
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
F4 = np.concatenate([E2M1, -E2M1])


def e4m3_table() -> np.ndarray:
    v = np.empty(256)
    for i in range(256):
        e, f = (i >> 3) & 15, i & 7
        m = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[i] = np.nan if (i & 127) == 127 else (-m if i & 128 else m)
    return v


F8 = e4m3_table()


def random_entries(rng, n):
    """codes [n, 256] and scales [n, 32] of plausible entries (scale about 1/3, any code)."""
    codes = rng.integers(0, 256, (n, 256)).astype(np.uint8)
    scales = rng.integers(0x20, 0x30, (n, 32)).astype(np.uint8)  # E4M3 0.125 .. 0.47
    return codes, scales


def decode(codes, scales):
    x = np.empty(codes.shape[:-1] + (D,))
    x[..., 0::2], x[..., 1::2] = F4[codes & 15], F4[codes >> 4]
    return x * np.repeat(F8[scales], 16, -1)


def norm_rope_q(q, weight, eps, pos, base):
    q = q.astype(np.float64)
    if weight is not None:
        q = weight * q / np.sqrt((q ** 2).mean(-1, keepdims=True) + eps)
    if pos is not None:
        q = np.concatenate([q[:, :448], rotate(q[:, 448:], pos, base)], -1)
    return q


def rotate(x, pos, base):
    t = float(pos) * base ** (-np.arange(32) / 32)
    c, s = np.cos(t), np.sin(t)
    a, b = x[:, 0::2], x[:, 1::2]
    out = np.empty_like(x)
    out[:, 0::2], out[:, 1::2] = a * c - b * s, a * s + b * c
    return out


def attention(x, q, scale, sink=None, q_rounded=False, pos=None, base=10000.0):
    """(out, lse, bound) of one query over rows x [n, 512]: float64 q [64, 512] already normalised and
    rotated; `bound` [64, 512] is what the kernel's output may be off before its own rounding.

    Roundings: P to f16, at most 2^-11 of each p, and O / l of each part of the rows to f16, at most 2^-11
    of sum p |x| over its rows, which with the parts' weights adds up to 2^-11 of the whole (a p below f16's smallest normal loses at most 2^-25
    absolutely against a row's maximum of at least e^-8: below 2^-13 relative to it, and n of them
    n 2^-13 2^-11 at most, kept in the term with max |x|); a logit is off by e_z = scale * sum |q x| *
    (2^-16 for at most 512 fp32 sums of 2^-24 and the staging, + 2^-11 where q was rounded to f16 after
    its normalisation or rotation), which moves every p by at most e_z relatively, and the denominator
    too; the fp32 sums of p x and of p add 2^-14 (chains of at most 1024 additions of 2^-24: one for 16 rows
    of a part, then the parts)."""
    n = x.shape[0]
    z = scale * (q @ x.T) if n else np.zeros((H, 0))
    top = z.max(1) if n else np.full(H, -np.inf)
    if sink is not None:
        top = np.maximum(top, sink)
    if not n and sink is None:
        return np.zeros((H, D)), np.full(H, -np.inf), np.zeros((H, D)), np.zeros(H)
    p = np.exp(z - top[:, None])
    den = p.sum(1) + (np.exp(sink - top) if sink is not None else 0.0)
    o = (p / den[:, None]) @ x if n else np.zeros((H, D))
    lse = top + np.log(den)
    if not n:
        return o, lse, np.zeros((H, D)), np.full(H, 2.0 ** -20)
    zx = scale * (np.abs(q) @ np.abs(x).T).max(1)
    ez = zx * (2.0 ** -16 + (2.0 ** -11 if q_rounded else 0.0)) + 2.0 ** -20
    mass = (p / den[:, None]) @ np.abs(x)
    bound = mass * (2.0 ** -11 + 2.0 ** -11 + 2 * ez[:, None] + 2.0 ** -14) + n * 2.0 ** -24 * np.abs(x).max()
    if pos is not None:  # the output turns back: pairs mix
        o = np.concatenate([o[:, :448], rotate(o[:, 448:], -pos, base)], -1)
        pair = bound[:, 448:].reshape(H, 32, 2).sum(-1, keepdims=True)
        bound[:, 448:] = np.broadcast_to(pair, (H, 32, 2)).reshape(H, 64) + 2.0 ** -20 * np.abs(x).max()
    # the lse: the logits' error of the fp32 sums, and the fp32 sum of probabilities (2^-14).  The rounding of q
    # to f16, by which a logit is off by e at most, is corrected in the first order: left are the square of its
    # width 2 e over 8, and of the correction e 2^-11 for its f16 terms and e 2^-9 for the output in it
    e = zx * 2.0 ** -11 if q_rounded else 0.0
    return o, lse, bound, zx * 2.0 ** -16 + e * e / 2 + e * (2.0 ** -11 + 2.0 ** -9) + 2.0 ** -14 + 2.0 ** -22 * np.abs(lse)


class PagedState:
    """Python model of csa2_page_tables."""

    def __init__(self, B, page, max_pages, n_pages, free):
        self.B, self.P, self.max_pages, self.n_pages = B, page, max_pages, n_pages
        self.have = [0] * B
        self.table = [[-1] * max_pages for _ in range(B)]
        self.free = list(free) + [-1] * (n_pages - len(free))
        self.n_free = len(free)

    def step(self, new, kept, m, n_rows):
        """Applies one call; returns (rows, row_start), or an error's status and detail."""
        P = self.P
        pages = lambda n: -(-n // P)  # noqa: E731
        for b in range(self.B):
            t = self.have[b] + new[b]
            if t < 0 or t > self.max_pages * P or kept[b] < 0:
                return 6, b
        rows = sum(max(x, 0) for x in new)
        if n_rows is not None and rows > n_rows:
            return 6, rows
        back = []
        for b in range(self.B):
            if new[b] < 0:
                pc = pages(self.have[b])
                for p in range(max(pages(self.have[b] + new[b]), min(kept[b], pc)), pc):
                    back.append(self.table[b][p])
        if self.n_free + len(back) > self.n_pages:
            return 6, self.n_free
        need = sum(pages(self.have[b] + new[b]) - pages(self.have[b]) for b in range(self.B) if new[b] >= 0)
        if need > self.n_free + len(back):
            return 7, need - self.n_free - len(back)
        stack = self.free[:self.n_free] + back
        for i, page in enumerate(back):
            self.free[self.n_free + i] = page
        out, start = [], [0]
        for b in range(self.B):
            if new[b] >= 0:
                for p in range(pages(self.have[b]), pages(self.have[b] + new[b])):
                    self.table[b][p] = stack.pop()
                for e in range(self.have[b], self.have[b] + new[b]):
                    out.append((b, self.table[b][e // P], e % P, e * m))
            self.have[b] += new[b]
            start.append(len(out))
        self.n_free = len(stack)
        return out, start


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
