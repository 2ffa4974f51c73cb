"""csa2_rope against the rotation in float64: layouts, parts of the head, scalings, types, strides and alignments, far
and negative positions, the gradient, streams and graphs.

The bound.  The angle of a position is off by |pos| 2^-53 turns twice (the reference's too, with theta's own rounding):
|pos| 2^-50 with the factor 2 pi; it is rounded to fp32 as a part of half a turn (pi 2^-25), cut at 2^-32 turns, and the
sine and cosine are off by 2 units of 2^-24 and multiplied by magnitude (2^-24); the two products and their sum add 2^-24
each: 2^-21 of |a| + |b| in all.  Then the output's own rounding."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from rotary_common import partners, rotate

pytestmark = pytest.mark.gpu

SCALINGS = {None: None, "linear": ("linear", 4.0), "yarn": ("yarn", 16.0, 65536, 32.0, 1.0)}


def scaling_of(name):
    s = SCALINGS[name]
    if s is None:
        return None
    return csa2.rope_scaling(csa2.SCALE_LINEAR, s[1]) if name == "linear" else csa2.rope_scaling(csa2.SCALE_YARN, *s[1:])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check(got, x, pos, n_rot, first, halves, scaling=None, inverse=False, magnitude=1.0, base=10000.0):
    """got, x: tensors [rows, heads, dim]; pos: int64 array."""
    x64 = x.detach().cpu().double().numpy()
    want = rotate(x64, pos, n_rot, first, halves, base, SCALINGS[scaling], inverse, magnitude)
    off = np.abs(got.detach().cpu().double().numpy() - want)
    far = np.abs(pos).astype(np.float64).reshape(-1, 1, 1) * 2.0 ** -50
    bound = partners(x64, n_rot, first, halves) * abs(magnitude) * (2.0 ** -21 + far)
    bound += (np.abs(want) + bound) * torch.finfo(x.dtype).eps / 2
    rest = np.ones(x.shape[-1], bool)
    rest[first:first + n_rot] = False
    assert (off <= bound).all(), (off / np.maximum(bound, 1e-300)).max()
    assert (off[..., rest] == 0).all()


def tensor(rng, shape, dtype):
    return to_dev(rng.standard_normal(shape).astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("rows,heads,dim,first,n_rot,scaling", [
    (1, 1, 2, 0, 2, None), (1, 64, 512, 448, 64, "yarn"), (3, 5, 96, 0, 48, "linear"), (129, 32, 128, 64, 64, "yarn"),
    (1000, 1, 512, 448, 64, None), (17, 2, 64, 0, 64, "yarn"), (2, 3, 20, 7, 6, "linear"), (5, 1, 1030, 3, 512, "yarn"),
    (4097, 1, 8, 0, 8, None), (40, 100, 64, 32, 32, "yarn")])
def test_rotation(rows, heads, dim, first, n_rot, scaling, halves, dtype):
    rng = np.random.default_rng(rows * dim + n_rot)
    x = tensor(rng, (rows, heads, dim), dtype)
    pos = rng.integers(0, 1 << 20, rows)
    pos[0] = 0
    rot = csa2.rotary(n_rot, first, int(halves), scaling=scaling_of(scaling))
    out = torch.full_like(x, 777.0)
    csa2.rope(x, rows, heads, dim, to_dev(pos), rot, out)
    check(out, x, pos, n_rot, first, halves, scaling)
    assert torch.equal(out[0], x[0])  # position 0
    # in place: the same bits
    y = x.clone()
    csa2.rope(y, rows, heads, dim, to_dev(pos), rot, y)
    assert torch.equal(y, out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_far_and_negative_positions_and_magnitude(inverse, halves, dtype):
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, -1, 1 << 20, -(1 << 20) - 7, (1 << 31) + 11, 1 << 40, -(1 << 45) + 3], np.int64)
    x = tensor(rng, (len(pos), 3, 128), dtype)
    rot = csa2.rotary(64, 32, int(halves), base=500000.0, magnitude=1.25)
    out = torch.empty_like(x)
    csa2.rope(x, len(pos), 3, 128, to_dev(pos), rot, out, inverse=inverse)
    check(out, x, pos, 64, 32, halves, None, inverse, 1.25, 500000.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("shift,gap,order", [(0, 64, "rows"), (0, 7, "rows"), (1, 0, "rows"), (8, 16, "heads"), (3, 5, "heads"),
                                             (4, 4, "rows")])
def test_strides_and_alignment(shift, gap, order, halves, dtype):
    rows, heads, dim = 37, 6, 128
    rng = np.random.default_rng(shift + gap)
    pos = rng.integers(0, 1 << 18, rows)
    rot = csa2.rotary(64, 64, int(halves))

    def strided(fill):
        if order == "rows":
            n, st = rows * (heads * dim + gap), (heads * dim + gap, dim, 1)
        else:
            n, st = heads * (rows * dim + gap), (dim, rows * dim + gap, 1)
        buf = torch.full((n + shift,), fill, dtype=dtype, device="cuda")
        return buf, buf.as_strided((rows, heads, dim), st, shift)

    (bx, x), (by, out) = strided(1.0), strided(777.0)
    x.copy_(tensor(rng, (rows, heads, dim), dtype))
    csa2.rope(x, rows, heads, dim, to_dev(pos), rot, out)
    check(out, x, pos, 64, 64, halves)
    other = torch.empty((rows, heads, dim), dtype=dtype, device="cuda")
    csa2.rope(x, rows, heads, dim, to_dev(pos), rot, other)  # strided in, dense out
    assert torch.equal(other, out)
    # nothing between the vectors is written
    was = out.clone()
    out.fill_(777.0)
    assert (by == 777.0).all()
    out.copy_(was)
    csa2.rope(x, rows, heads, dim, to_dev(pos), rot, x)
    assert torch.equal(x, out) and bx.isfinite().all()


def test_heads_that_share_one_vector():
    # a broadcast input: stride 0 over heads
    rng = np.random.default_rng(3)
    x, pos = tensor(rng, (9, 1, 64), torch.bfloat16), rng.integers(0, 1000, 9)
    out = torch.empty((9, 4, 64), dtype=torch.bfloat16, device="cuda")
    csa2.rope(x.expand(9, 4, 64), 9, 4, 64, to_dev(pos), csa2.rotary(64), out)
    check(out, x.expand(9, 4, 64), pos, 64, 0, False)


@pytest.mark.parametrize("halves", [False, True])
def test_gradient_is_the_inverse(halves):
    # y = R x: the rows of the Jacobian, from unit vectors and from differences, against R^T g
    dim, n_rot, first = 24, 16, 4
    rng = np.random.default_rng(9)
    p = to_dev(np.full(dim, 12345))
    rot = csa2.rotary(n_rot, first, int(halves), magnitude=1.5)
    eye, jac = torch.eye(dim, device="cuda"), torch.empty((dim, dim), device="cuda")
    csa2.rope(eye.view(dim, 1, dim), dim, 1, dim, p, rot, jac.view(dim, 1, dim))  # jac[i] = R e_i
    g = tensor(rng, (1, 1, dim), torch.float32)
    dx = torch.empty_like(g)
    csa2.rope(g, 1, 1, dim, p[:1], rot, dx, inverse=True)
    want = jac.double() @ g.double().flatten()
    # both sides: 2^-21 of the pair's |g|, times magnitude
    assert ((dx.double().flatten() - want).abs() <= 2 * 1.5 * 2.0 ** -21 * g.abs().sum()).all()
    x = tensor(rng, (1, 1, dim), torch.float32)
    loss = lambda v: _loss(v, g, p[:1], rot, dim)  # noqa: E731
    h = 0.5  # the loss is linear: any step will do
    for c in range(dim):
        up, down = x.clone(), x.clone()
        up[..., c] += h
        down[..., c] -= h
        step = (up[..., c] - down[..., c]).double().item()
        slope = (loss(up) - loss(down)) / step
        # each loss: 2^-21 1.5 (|a| + |b|) |g| summed over the channels
        bound = 4 * 2.0 ** -21 * 1.5 * (2 * (x.abs().max() + h) * g.abs().sum()).item() / step
        assert abs(slope - dx[0, 0, c].double().item()) <= bound


def _loss(v, g, p, rot, dim):
    y = torch.empty_like(v)
    csa2.rope(v, 1, 1, dim, p, rot, y)
    return (y.double() * g.double()).sum().item()


def test_indexer_queries_rotated_then_quantized():
    # as a decode step runs them: rotation, then the MXFP4 query
    B = 5
    rng = np.random.default_rng(2)
    q, pos = tensor(rng, (B, 32, 128), torch.bfloat16), rng.integers(0, 1 << 20, B)
    rot = csa2.rotary(64, 64, csa2.ROPE_HALVES, scaling=scaling_of("yarn"))
    turned, out = torch.empty_like(q), torch.empty_like(q)
    csa2.rope(q, B, 32, 128, to_dev(pos), rot, turned)
    csa2.quantize_index_query(turned, B * 32, out)
    check(turned, q, pos, 64, 64, True, "yarn")
    group = turned.float().view(-1, 32)
    # half a step of the largest binade: 2^(e - 2), e of the largest value, is at most a quarter of it
    assert ((out.float().view(-1, 32) - group).abs() <= group.abs().amax(1, keepdim=True) / 4).all()


def test_streams_graph_and_no_rows():
    rng = np.random.default_rng(4)
    x, pos = tensor(rng, (300, 8, 128), torch.bfloat16), rng.integers(0, 1 << 20, 300)
    d, rot = to_dev(pos), csa2.rotary(128, 0, csa2.ROPE_HALVES)
    want, out = torch.empty_like(x), torch.empty_like(x)
    csa2.rope(x, 300, 8, 128, d, rot, want)
    csa2.rope(x, 0, 8, 128, d, rot, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    csa2.rope(x, 300, 8, 128, d, rot, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.rope(x, 300, 8, 128, d, rot, out)
    x.copy_(tensor(rng, (300, 8, 128), torch.bfloat16))
    d.copy_(to_dev(rng.integers(0, 1 << 20, 300)))
    graph.replay()
    csa2.rope(x, 300, 8, 128, d, rot, want)
    assert torch.equal(out, want)


@pytest.mark.parametrize("halves", [False, True])
def test_angles_of_slow_pairs_at_far_positions(halves):
    # an angle is off by |pos| (3 theta / 2 pi 2^-53 + 2^-65) turns (the power's, the quotient's and 2 pi's rounding of
    # theta, and the fraction's own): beside the angle in 50 digits, which numpy's doubles do not have
    getcontext().prec = 50
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582")
    pos, n, base = np.array([1 << 50, -(1 << 50) - 12345, (1 << 51) + 7, 3 << 48], np.int64), 64, 1e9
    turns = [(Decimal(base).ln() * Decimal(-2 * i) / n).exp() / two_pi for i in range(n // 2)]
    angle = np.array([[float((int(p) * t) % 1 * two_pi) for t in turns] for p in pos])
    x = np.zeros((len(pos), 1, n), np.float32)
    a, b = (np.arange(n // 2), np.arange(n // 2, n)) if halves else (np.arange(0, n, 2), np.arange(1, n, 2))
    x[:, :, a] = 1.0
    out = torch.empty(x.shape, device="cuda")
    csa2.rope(to_dev(x), len(pos), 1, n, to_dev(pos), csa2.rotary(n, 0, int(halves), base=base), out)
    got = out.cpu().double().numpy()[:, 0]
    off = np.abs(pos).astype(np.float64)[:, None] * (3 * np.array([float(t) for t in turns]) * 2.0 ** -53 + 2.0 ** -65)
    bound = 2 * np.pi * off + 2.0 ** -21 + 2.0 ** -24
    for have, want in ((got[:, a], np.cos(angle)), (got[:, b], np.sin(angle))):
        assert (np.abs(have - want) <= bound).all(), (np.abs(have - want) / bound).max()
