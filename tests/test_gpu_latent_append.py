"""csa2_latent_append: the bytes are those of the cache's codec on the latents normalised and rotated in float64 and
rounded to fp32 once.

Bytes have to be equal: a value is off by at most 2^-36 of its vector's largest, so it is rounded to another fp32 than
the reference's with a chance of about 2^-12, and that one lies beside a border of the codec with 2^-22."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from rotary_common import rotate

pytestmark = pytest.mark.gpu
YARN = ("yarn", 16.0, 65536, 32.0, 1.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Pool:
    """Planes of n_slots pages of P entries, all bytes 0xA5."""

    def __init__(self, n_slots, P):
        self.n_slots, self.P = n_slots, P
        self.planes = csa2.Planes.empty(n_slots, P)
        for t in self.parts:
            t.fill_(0xA5)

    @property
    def parts(self):
        p = self.planes
        return p.kv_codes, p.kv_scales, p.ix_codes, p.ix_scales

    def bytes(self):
        return [t.cpu().numpy() for t in self.parts]


def reference(oracle, x, key, weight, eps, pos, rope, scaling, key_rot):
    """The four planes' rows of latents x and keys (float64 of what the call is given)."""
    out = [None] * 4
    if x is not None:
        y = x
        if weight is not None:
            y = weight.astype(np.float64) * y / np.sqrt((y ** 2).mean(-1, keepdims=True) + float(np.float32(eps)))
        if rope:
            y = rotate(y, pos, 64, 448, False, 10000.0, scaling)
        out[:2] = oracle.quantize_main(np.ascontiguousarray(y.astype(np.float32)))
    if key is not None:
        k = rotate(key, pos, *key_rot) if key_rot else key
        out[2:] = oracle.quantize_index(np.ascontiguousarray(k.astype(np.float32)))
    return out


def run(oracle, R, P=16, seed=0, dtype=torch.float32, norm=True, rope=True, scaling=YARN, key_rot=(64, 64, True, 10000.0),
        parts="both", eps=1e-6, scale=1.0, graph=False, positions=None):
    rng = np.random.default_rng(seed)
    pages = -(-R // P) + 2
    pool = Pool(pages, P)
    at = rng.permutation(pages * P)[:R]
    slot, entry = (at // P).astype(np.int32), (at % P).astype(np.int64)
    pos = rng.integers(0, 1 << 20, R) if positions is None else positions
    x = (to_dev((scale * rng.standard_normal((R, 512))).astype(np.float32)).to(dtype)) if parts != "key" else None
    key = to_dev(rng.standard_normal((R, 128)).astype(np.float32)).to(dtype) if parts != "x" else None
    weight = (1 + 0.3 * rng.standard_normal(512)).astype(np.float32) if norm else None
    sc = csa2.rope_scaling(csa2.SCALE_YARN, *scaling[1:]) if scaling else None
    nr = csa2.norm_rope(to_dev(weight) if norm else None, eps, rope) if norm or rope else None
    rot = csa2.rotary(key_rot[0], key_rot[1], int(key_rot[2]), key_rot[3]) if key_rot else None
    ws = csa2.workspace(csa2.latent_append_workspace_size(R))
    ws.fill_(0xFF)
    args = (x, R, pool.planes, pages, to_dev(slot), to_dev(entry), ws)
    kw = dict(key=key, kv_nr=nr, scaling=sc, pos=to_dev(pos) if rope or key_rot else None, key_rot=rot)
    csa2.latent_append(*args, **kw)
    assert csa2.check(ws) == (0, 0)
    f = lambda t: None if t is None else t.cpu().double().numpy()  # noqa: E731
    want = reference(oracle, f(x), f(key), weight, eps, pos, rope, scaling, key_rot)
    rest = np.setdiff1d(np.arange(pages * P), at)
    for got, w in zip(pool.bytes(), want):
        assert (got[rest] == 0xA5).all()
        if w is None:
            assert (got == 0xA5).all()
        else:
            assert np.array_equal(got[at], w), np.argwhere(got[at] != w)[:5]
    return args, kw, pool


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm,rope", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("R", [1, 3, 131, 2000])
def test_bytes(oracle_mod, R, norm, rope, dtype):
    run(oracle_mod, R, seed=R, dtype=dtype, norm=norm, rope=rope)


def test_bytes_of_many_rows(oracle_mod):
    # about a thousand of them have a value whose fp32 form lies too near a border of the codec
    run(oracle_mod, 20000, P=64, seed=21)
    run(oracle_mod, 20000, P=64, seed=22, norm=False, dtype=torch.bfloat16)


@pytest.mark.parametrize("R", [511, 513, 11999, 12000, 12001])
def test_bytes_where_the_form_changes(oracle_mod, R):
    run(oracle_mod, R, P=64, seed=R)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm,rope", [(True, True), (False, True), (True, False), (False, False)])
def test_bytes_of_two_rows_a_warp(oracle_mod, norm, rope, dtype):
    run(oracle_mod, 12003, P=64, seed=30, dtype=dtype, norm=norm, rope=rope, parts="x")


@pytest.mark.parametrize("scale,eps", [(1e-18, 1e-6), (1e-15, 0.0), (1e30, 1e-6)])
def test_many_rows_far_from_one(oracle_mod, scale, eps):
    run(oracle_mod, 12001, P=64, seed=31, scale=scale, eps=eps, parts="x")


def test_many_rows_of_which_some_are_not_written(oracle_mod):
    # padding, destinations outside and a NaN beside rows that share a warp with them
    R, P = 12005, 64
    rng = np.random.default_rng(32)
    x = rng.standard_normal((R, 512)).astype(np.float32)
    pages = -(-R // P)
    at = rng.permutation(R)
    slot, entry = (at // P).astype(np.int32), (at % P).astype(np.int64)
    pad, out, nan = [0, 5, 77, R - 1], [2, 101, 5001], [9, 200, 6000, 6001]
    slot[pad], entry[pad] = -1, -1
    slot[out] = pages
    x[nan, 100] = np.nan
    weight = (1 + 0.3 * rng.standard_normal(512)).astype(np.float32)
    pos = rng.integers(0, 1 << 20, R)
    pool, ws = Pool(pages, P), csa2.workspace(256)
    csa2.latent_append(to_dev(x), R, pool.planes, pages, to_dev(slot), to_dev(entry), ws,
                       kv_nr=csa2.norm_rope(to_dev(weight), 1e-6, True), pos=to_dev(pos))
    assert csa2.check(ws) == (6, pages)
    clean = np.where(np.isfinite(x), x, 0).astype(np.float64)
    want = reference(oracle_mod, clean, None, weight, 1e-6, pos, True, None, None)
    good = np.setdiff1d(np.arange(R), pad + out + nan)
    for got, w in zip(pool.bytes(), want[:2]):
        assert np.array_equal(got[at[good]], w[good])
        assert (got[at[pad + out]] == 0xA5).all()


@pytest.mark.parametrize("key_rot", [None, (128, 0, False, 10000.0), (128, 0, True, 500000.0), (2, 126, False, 10000.0),
                                     (48, 5, True, 10000.0), (64, 0, False, 10000.0)])
def test_keys(oracle_mod, key_rot):
    run(oracle_mod, 77, seed=1, key_rot=key_rot)


@pytest.mark.parametrize("parts", ["x", "key"])
def test_either_half_alone(oracle_mod, parts):
    run(oracle_mod, 40, seed=2, parts=parts)


@pytest.mark.parametrize("scale,eps", [(1e-18, 1e-6), (1e-15, 0.0), (3e17, 1e-6), (1e30, 1e-6), (1e-3, 1e30)])
def test_rows_far_from_one(oracle_mod, scale, eps):
    run(oracle_mod, 33, seed=3, scale=scale, eps=eps)


def test_positions(oracle_mod):
    pos = np.array([0, 1, -1, 7, -123456, 1 << 20, (1 << 21) + 1, 65536])
    run(oracle_mod, len(pos), seed=4, positions=pos, scaling=None)


def test_zeros_keep_their_sign_and_scales_of_zero(oracle_mod):
    R, P = 3, 8
    x = np.zeros((R, 512), np.float32)
    x[1, ::3], x[1, 1::3], x[1, 2::3] = -0.0, 1.0, 0.0
    x[2, :16] = 1e-8  # a scale that rounds to zero
    key = np.zeros((R, 128), np.float32)
    key[1, 5], key[1, 6] = -0.0, 3.0
    pool, ws = Pool(1, P), csa2.workspace(256)
    csa2.latent_append(to_dev(x), R, pool.planes, 1, to_dev(np.zeros(R, np.int32)), to_dev(np.arange(R)), ws, key=to_dev(key))
    plain = Pool(1, P)
    csa2.quantize_entries(plain.planes, to_dev(x), to_dev(key), R, 0)
    for a, b in zip(pool.bytes(), plain.bytes()):
        assert np.array_equal(a, b)


def test_of_what_is_not_finite_the_rest_stays(oracle_mod):
    # an infinity or NaN stays in its groups of the main copy, and in its row
    R, P = 4, 4
    rng = np.random.default_rng(8)
    x = rng.standard_normal((R, 512)).astype(np.float32)
    x[1, 40], x[2, 500] = np.inf, np.nan
    pos, ws = np.arange(R) + 5, csa2.workspace(256)
    pool, slot, entry = Pool(1, P), to_dev(np.zeros(R, np.int32)), to_dev(np.arange(R))
    nr = csa2.norm_rope(None, 1e-6, True)
    csa2.latent_append(to_dev(x), R, pool.planes, 1, slot, entry, ws, kv_nr=nr, pos=to_dev(pos))
    assert csa2.check(ws) == (0, 0)
    clean = np.where(np.isfinite(x), x, 0).astype(np.float32)
    codes, scales = reference(oracle_mod, clean.astype(np.float64), None, None, 0, pos, True, None, None)[:2]
    got = pool.bytes()
    same = np.ones((R, 32), bool)
    same[1, 2] = same[2, 31] = False
    assert np.array_equal(got[1][same], scales[same])
    assert np.array_equal(got[0].reshape(R, 32, 8)[same], codes.reshape(R, 32, 8)[same])


def test_padding_and_rows_outside(oracle_mod):
    R, P = 6, 8
    rng = np.random.default_rng(6)
    x, key = to_dev(rng.standard_normal((R, 512)).astype(np.float32)), to_dev(rng.standard_normal((R, 128)).astype(np.float32))
    slot, entry = np.array([0, -1, 2, 1, -1, 1], np.int32), np.array([1, -1, 7, 0, -1, 3], np.int64)
    ws = csa2.workspace(256)

    def append(s, e):
        pool = Pool(3, P)
        csa2.latent_append(x, R, pool.planes, 3, to_dev(s), to_dev(e), ws, key=key)
        return csa2.check(ws), pool.bytes()

    status, got = append(slot, entry)
    assert status == (0, 0)
    for s, e, detail in ((-1, 3, -1), (1, -1, -1), (3, 0, 3), (0, P, P), (0, -5, -5), (-2, -1, -2)):
        bad_s, bad_e = slot.copy(), entry.copy()
        bad_s[1], bad_e[1] = s, e
        status, other = append(bad_s, bad_e)
        assert status == (6, detail)
        for a, b in zip(got, other):
            assert np.array_equal(a, b)  # the others are written, the bad one nowhere


def test_graph_with_a_moving_map(oracle_mod):
    args, kw, pool = run(oracle_mod, 50, seed=11)
    want = pool.bytes()
    for t in pool.parts:
        t.fill_(0xA5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.latent_append(*args, **kw)
    graph.replay()
    for a, b in zip(want, pool.bytes()):
        assert np.array_equal(a, b)
    args[4].fill_(-1)  # a step with nothing to append
    args[5].fill_(-1)
    for t in pool.parts:
        t.fill_(0x5A)
    graph.replay()
    assert csa2.check(args[6]) == (0, 0)
    assert all((b == 0x5A).all() for b in pool.bytes())


def test_no_rows():
    pool, ws = Pool(1, 4), csa2.workspace(256)
    ws.fill_(0xFF)
    csa2.latent_append(None, 0, pool.planes, 1, None, None, ws)
    assert csa2.check(ws) == (0, 0)
