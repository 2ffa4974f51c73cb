"""csa2_latent_append on values at the ends of fp32.  The bytes are the codec's (csa2_quantize_entries) on the values of the
definition."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from rotary_common import rotate
from test_gpu_latent_append import Pool, reference

pytestmark = pytest.mark.gpu
INF, NAN = np.inf, np.nan
ODD = [INF, -INF, NAN]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def append(x, key, R, **kw):
    """The four planes' rows, row r at entry r."""
    pool, ws = Pool(1, R), csa2.workspace(256)
    csa2.latent_append(x, R, pool.planes, 1, torch.zeros(R, dtype=torch.int32, device="cuda"), torch.arange(R, device="cuda"), ws,
                       key=key, **kw)
    assert csa2.check(ws) == (0, 0)
    return pool.bytes()


def codec(x, key, R):
    pool = Pool(1, R)
    csa2.quantize_entries(pool.planes, x.float(), key.float(), R, 0)
    return pool.bytes()


def with_odd_values(R, dtype):
    """Rows of which all but every fifth have infinities and NaN: one, two of both signs, next to a NaN, in both ends."""
    rng = np.random.default_rng(R)
    x, key = rng.standard_normal((R, 512)).astype(np.float32), rng.standard_normal((R, 128)).astype(np.float32)
    for v in (x, key):
        n = v.shape[1]
        for r in range(R):
            for _ in range(r % 5):
                v[r, rng.integers(0, n)] = ODD[rng.integers(0, 3)]
        v[1, 3], v[2, n - 1], v[3, [0, 5]] = INF, -INF, (NAN, INF)
    return to_dev(x).to(dtype), to_dev(key).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [7, 12003])
def test_what_is_not_finite_has_the_codecs_bytes(R, dtype):
    x, key = with_odd_values(R, dtype)
    for a, b in zip(append(x, key, R), codec(x, key, R)):
        assert np.array_equal(a, b), np.argwhere(a != b)[:5]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [7, 12003])
def test_groups_beside_a_rotation_keep_theirs(R, dtype):
    # the last 64 channels of the main copy turn, and of the key: the others' groups are the codec's
    x, key = with_odd_values(R, dtype)
    got = append(x, key, R, kv_nr=csa2.norm_rope(None, 1e-6, True), key_rot=csa2.rotary(64, 64),
                 pos=torch.arange(R, device="cuda") + 3)
    for a, b, n in zip(got, codec(x, key, R), (224, 28, 32, 2)):
        assert np.array_equal(a[:, :n], b[:, :n]), np.argwhere(a[:, :n] != b[:, :n])[:5]


@pytest.mark.parametrize("R", [5, 12001])
@pytest.mark.parametrize("scale,eps,gain", [(1e-20, 1e4, 1e22), (1e-25, 1e12, 1e31), (1e-30, 0.5, 1e30), (1e-13, 2e3, 1e15)])
def test_small_rows_that_eps_outweighs(oracle_mod, R, scale, eps, gain):
    rng = np.random.default_rng(R)
    x = (scale * rng.standard_normal((R, 512))).astype(np.float32)
    weight = (gain * (1 + 0.3 * rng.standard_normal(512))).astype(np.float32)
    pos = rng.integers(0, 1 << 20, R)
    got = append(to_dev(x), None, R, kv_nr=csa2.norm_rope(to_dev(weight), eps, True), pos=to_dev(pos))
    want = reference(oracle_mod, x.astype(np.float64), None, weight, eps, pos, True, None, None)
    assert (want[0] != 0).mean() > 0.5
    for a, b in zip(got[:2], want[:2]):
        assert np.array_equal(a, b), np.argwhere(a != b)[:5]


@pytest.mark.parametrize("halves", [False, True])
def test_pairs_that_turn_past_the_largest_value(halves):
    # (a, a) turned by an eighth of a turn is 1.41 a: an infinity as fp32, its partner nearly nothing
    R = 64
    rng = np.random.default_rng(4)
    x = rng.standard_normal((R, 512)).astype(np.float32)
    key = rng.standard_normal((R, 128)).astype(np.float32)
    x[:, 448:] = 3e38 * rng.choice([-1, 1], (R, 64))
    key[:, 64:] = 3e38 * rng.choice([-1, 1], (R, 64))
    pos = rng.integers(0, 1 << 20, R)
    got = append(to_dev(x), to_dev(key), R, kv_nr=csa2.norm_rope(None, 1e-6, True), key_rot=csa2.rotary(64, 64, int(halves)),
                 pos=to_dev(pos))
    with np.errstate(over="ignore"):
        turned = [rotate(x.astype(np.float64), pos, 64, 448, False, 10000.0).astype(np.float32),
                  rotate(key.astype(np.float64), pos, 64, 64, halves, 10000.0).astype(np.float32)]
    assert all(np.isinf(t).any(1).mean() > 0.9 for t in turned)
    for a, b in zip(got, codec(to_dev(turned[0]), to_dev(turned[1]), R)):
        assert np.array_equal(a, b), np.argwhere(a != b)[:5]
