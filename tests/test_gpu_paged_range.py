"""Paged and shared-prefix attention where a worst-case bound of random data would hide a fault: a long context
far behind one strong row, and rows that can be counted in the output, so that none is lost, read twice or
weighted wrongly wherever it lies."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from paged_common import D, H

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def attend(codes, scales, P, table, n, q, groups=None, shared=(), shared_max=0, own_max=0, dtype=torch.float32):
    """paged_attn_decode, or with groups prefix_attn_decode: (out, lse)."""
    N, B = codes.shape[0], len(n)
    ix = torch.empty((N, 64), dtype=torch.uint8, device="cuda"), torch.empty((N, 4), dtype=torch.uint8, device="cuda")
    planes, pages = csa2.Planes(codes, scales, *ix, P), csa2.pages(table, N // P)
    counts = to_dev(np.asarray(n, np.int32))
    out = torch.full((B, H, D), 777.0, dtype=dtype, device="cuda")
    lse = torch.full((B, H), 777.0, dtype=torch.float32, device="cuda")
    if groups is None:
        ws = csa2.workspace(csa2.paged_attn_workspace_size(B, max(n), 0))
        csa2.paged_attn_decode(planes, pages, B, counts, max(n), None, 0, q, SCALE, out, ws, lse_out=lse)
    else:
        start, shared = to_dev(np.asarray(groups, np.int32)), to_dev(np.asarray(shared, np.int32))
        ws = csa2.workspace(csa2.prefix_attn_workspace_size(B, len(groups) - 1, shared_max, own_max, 0))
        csa2.prefix_attn_decode(planes, pages, B, counts, len(groups) - 1, start, shared, shared_max, own_max, None, 0,
                                q, SCALE, out, ws, lse_out=lse)
    assert csa2.check(ws) == (0, 0)
    return out, lse


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("at", [0, 63, 40_001, 65_535])
def test_rows_far_behind_one_add_up(prefix, at, dtype):
    """Row `at` is 1 in channels 0 .. 255 and 0 in the others, all other rows the opposite, and head h's query a_h
    and 0: the others' logits are 0, the strong row's z = 256 a_h / sqrt(512), from 6 to 25 nats above them.
    152 queries, so that a CTA (or pair) runs all rows of one.

    With w = e^-z: out = 1 / (1 + (n - 1) w) in the first half and (n - 1) w / (1 + (n - 1) w) in the second.
    Errors of the second half: each w is rounded to f16 (2^-11), moves by the logit's error e_z = z 2^-16 + 2^-20
    in numerator and denominator, fp32 sums add 2^-14, and of a weight at most 2^-36 of the strongest row's is
    lost.  A bf16 output is rounded by 2^-8 and its part by 2^-11 or 2^-29."""
    n, P, B = 65_536, 64, 152
    codes = np.zeros((n, 256), np.uint8)
    codes[:, 128:] = 0x22  # E2M1 code 2 is 1.0
    codes[at] = codes[at, ::-1]
    a = torch.linspace(0.5, 2.25, H).to(torch.bfloat16)
    q = torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, :256] = a.cuda()[None, :, None]
    table = to_dev(np.repeat(np.arange(n // P, dtype=np.int32)[None], B, 0))
    more = dict(groups=[0, B], shared=[n], shared_max=n) if prefix else {}
    more["dtype"] = dtype
    got = attend(to_dev(codes), to_dev(np.full((n, 32), 0x38, np.uint8)), P, table, [n] * B, q, **more)
    out, lse = (x.double().cpu().numpy() for x in got)
    z = a.double().numpy() * 256 * SCALE
    w = np.exp(-z)
    den = 1 + (n - 1) * w
    ez = z * 2.0 ** -16 + 2.0 ** -20
    rel = 2.0 ** -11 + 2 * ez + 2.0 ** -14
    lost = (n - 1) * np.minimum(w, 2.0 ** -36) / den
    if dtype == torch.bfloat16:
        rel = rel + (2.0 ** -8 + 2.0 ** -11) * (1 + 2.0 ** -8)
        lost = lost + 2.0 ** -29 * (1 + 2.0 ** -8)
    for half, want in ((out[..., :256], 1 / den), (out[..., 256:], (n - 1) * w / den)):
        err = np.abs(half - want[None, :, None]).max((0, 2))
        assert (err <= want * rel + lost).all(), (err / (want * rel + lost)).max()
    assert (np.abs(lse - (z + np.log(den))) <= ez + 2.0 ** -14).all()


class Counted:
    """A pool of entries, each 6.0 in one random channel, and sequences of its pages: with queries of zero every row
    weighs the same, and out[c] = 6 (rows of channel c) / (rows), some 128 rows a channel at 65,536.  The sums of
    probabilities and of products are whole multiples of one power of two, hence exact; left are a part's division,
    its weight and the sum of at most 152 parts, in fp32: 160 times 2^-24, less than 2^-16 of each channel's value,
    against 2^-8 or so for one row."""

    def __init__(self, seed, n_pages, P):
        rng = np.random.default_rng(seed)
        self.P, self.rng = P, rng
        self.channel = rng.integers(0, D, n_pages * P)
        codes = np.zeros((n_pages * P, 256), np.uint8)
        codes[np.arange(n_pages * P), self.channel // 2] = 7 << 4 * (self.channel % 2)
        self.codes, self.scales = to_dev(codes), torch.full((n_pages * P, 32), 0x38, dtype=torch.uint8, device="cuda")

    def counts(self, pages, n):
        j = np.arange(n)
        return np.bincount(self.channel[pages[j // self.P].astype(np.int64) * self.P + j % self.P], minlength=D)

    def check(self, table, n, out, lse, of=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(len(n)) if of is None else of:
            if n[b] == 0:
                assert not out[b].any() and np.isneginf(lse[b]).all()
                continue
            want = 6.0 * self.counts(table[b], n[b]) / n[b]
            assert (np.abs(out[b] - want) <= want * 2.0 ** -16).all(), b
            assert (np.abs(lse[b] - np.log(n[b])) <= 2.0 ** -20 + 2.0 ** -22 * np.log(n[b])).all(), b


@pytest.mark.parametrize("P", [16, 97])
@pytest.mark.parametrize("n", [[65_536], [65_537 - 1, 30_001, 0, 1, 63, 64, 65, 4_097],
                               [int(x) for x in np.random.default_rng(3).integers(0, 2_000, 300)]])
def test_paged_rows_are_counted(n, P):
    mp = -(-max(n) // P)
    c = Counted(1, mp + 7, P)
    table = np.stack([c.rng.permutation(mp + 7)[:mp] for _ in n]).astype(np.int32)
    q = torch.zeros((len(n), H, D), dtype=torch.bfloat16, device="cuda")
    c.check(table, n, *attend(c.codes, c.scales, P, to_dev(table), n, q))


@pytest.mark.parametrize("sizes,shared,own", [
    ([64], [65_000], 300),               # one group's image
    ([5] * 18, [65_536] * 18, 70),       # beyond 2^20 entries: the last groups' are widened where they are read
    ([7, 9, 5, 13], [4_001, 3_999, 65, 20_000], 600),
    ([31, 0, 1, 30], [3_000, 10, 4_500, 0], 2_000),
    ([2, 3], [9_000, 8_000], 300)])      # small groups: every query by itself
def test_prefix_rows_are_counted(sizes, shared, own):
    P, B = 64, sum(sizes) + 2            # and two queries outside the groups
    mp = -(-(max(shared) + own) // P)
    c = Counted(2, mp + 50, P)
    start = np.concatenate([[0], np.cumsum(sizes)])
    table, n = np.zeros((B, mp), np.int32), []
    for g, size in enumerate(sizes):
        lead = c.rng.permutation(mp + 50)[:mp]
        for b in range(start[g], start[g + 1]):
            table[b] = lead
            whole = shared[g] // P
            if shared[g] % P == 0:       # pages behind the shared ones are each query's own
                table[b, whole:] = c.rng.permutation(mp + 50)[:mp - whole]
            n.append(shared[g] + int(c.rng.integers(0, own + 1)))
        if size > 3:
            n[-2], n[-3] = shared[g] // 3, 0   # a query that sees a part of the prefix, and an empty one
    for b in (B - 2, B - 1):
        table[b] = c.rng.permutation(mp + 50)[:mp]
        n.append(min(own, 200))
    q = torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda")
    got = attend(c.codes, c.scales, P, to_dev(table), n, q, groups=start, shared=shared, shared_max=max(shared), own_max=own)
    c.check(table, n, *got)


def test_counting_notices_a_lost_row():
    # of 65,536 rows: one lost, one twice, the last 64 lost, one page for another
    c = Counted(4, 1100, 64)
    pages, n = np.arange(1024), 65_536
    full = c.counts(pages, n)
    tol = 6.0 * full / n * 2.0 ** -16
    for wrong, m in ((c.counts(pages, n - 1), n), (full + np.eye(D, dtype=int)[5], n), (c.counts(pages, n - 64), n),
                     (c.counts(np.r_[pages[:500], 1050, pages[501:]], n), n)):
        assert (np.abs(6.0 * wrong / m - 6.0 * full / n) > tol).any()


@pytest.mark.parametrize("sizes,shared,own", [([64], [4_000], 300), ([6, 5, 7, 20], [3_999, 0, 9_000, 700], 150)])
def test_pairs_give_the_same_bits_again_and_again(sizes, shared, own):
    # copies from the image, own rows and many queries to a pair of CTAs in turn, while another stream loads memory
    P, B = 16, sum(sizes)
    mp = -(-(max(shared) + own) // P)
    rng = np.random.default_rng(6)
    codes = to_dev(rng.integers(0, 256, ((mp + 9) * P, 256)).astype(np.uint8))
    scales = to_dev(rng.integers(0x20, 0x30, ((mp + 9) * P, 32)).astype(np.uint8))
    start = np.concatenate([[0], np.cumsum(sizes)])
    table = to_dev(np.concatenate([np.repeat(rng.permutation(mp + 9)[None, :mp], s, 0) for s in sizes]).astype(np.int32))
    n = [shared[g] + int(rng.integers(0, own + 1)) for g, s in enumerate(sizes) for _ in range(s)]
    q = torch.randn((B, H, D), device="cuda", generator=torch.Generator("cuda").manual_seed(6)).to(torch.bfloat16)
    more = dict(groups=start, shared=shared, shared_max=65_536 if B < 64 else max(shared), own_max=own)
    table = table if B >= 64 else torch.nn.functional.pad(table, (0, 65_536 // P - mp))
    first = attend(codes, scales, P, table, n, q, **more)
    other, noise = torch.cuda.Stream(), torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    for i in range(40):
        with torch.cuda.stream(other):
            noise.add_(1)
        out, lse = attend(codes, scales, P, table, n, q, **more)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), i


@pytest.mark.parametrize("shared_max,few", [(65_536, False), (4_000, True)])  # pairs, and every query by itself
@pytest.mark.parametrize("case", ["first", "ninth", "late", "last", "none", "ties", "empty"])
def test_whose_row_holds_the_shared_entries(case, shared_max, few):
    """Groups that begin with queries too short for the prefix: it is read through the first row that has all of it,
    else the longest (of equal ones the first).  Every other row ends with its own entries, in page ids that no pool
    has: reading through one of them would be reported."""
    P, sizes, want = 64, [300, 7, 1, 12] if not few else [30, 7, 1, 12], 1_000
    B = sum(sizes)
    start = np.concatenate([[0], np.cumsum(sizes)])
    c = Counted(5, 200, P)
    n, table = np.zeros(B, int), np.full((B, shared_max // P + 1), 0x7fffffff, np.int32)
    for g, size in enumerate(sizes):
        lead = c.rng.permutation(200)[:20]
        m = c.rng.integers(0, 900, size)
        at = {"first": 0, "ninth": min(8, size - 1), "late": size * 2 // 3, "last": size - 1}.get(case)
        if at is not None:
            m[at] = 1_100
            m[at + 1:] = c.rng.integers(0, 1_100, size - at - 1)
        if case == "ties":
            m[size // 2:] = 905
        if case == "empty":
            m[:] = 0
        n[start[g]:start[g + 1]] = m
        for b in range(start[g], start[g + 1]):
            table[b, :-(-n[b] // P)] = lead[:-(-n[b] // P)]
    q = torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda")
    got = attend(c.codes, c.scales, P, to_dev(table), n, q, groups=start, shared=[want] * 4, shared_max=shared_max, own_max=1_100)
    c.check(table, n, *got)
