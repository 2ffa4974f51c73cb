"""What many weak rows add up to: paged and shared-prefix attention where a long context lies far behind one
strong row."""
import numpy as np
import pytest

from gpu_common import csa2, require_gpu, to_dev, torch
from paged_common import D, H

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def attend(prefix, codes, scales, n, P, q, B):
    """The same call for B queries q[i] over the same n entries: (out, lse) in float64."""
    N = codes.shape[0]
    ix = torch.empty((N, 64), dtype=torch.uint8, device="cuda"), torch.empty((N, 4), dtype=torch.uint8, device="cuda")
    planes = csa2.Planes(to_dev(codes), to_dev(scales), *ix, P)
    table = to_dev(np.repeat(np.arange(N // P, dtype=np.int32)[None], B, 0))
    counts = to_dev(np.full(B, n, np.int32))
    out = torch.full((B, H, D), 777.0, dtype=torch.float32, device="cuda")
    lse = torch.full((B, H), 777.0, dtype=torch.float32, device="cuda")
    pages = csa2.pages(table, N // P)
    if prefix:
        start, shared = to_dev(np.array([0, B], np.int32)), to_dev(np.array([n], np.int32))
        ws = csa2.workspace(csa2.prefix_attn_workspace_size(B, 1, n, 0, 0))
        csa2.prefix_attn_decode(planes, pages, B, counts, 1, start, shared, n, 0, None, 0, q, SCALE, out, ws, lse_out=lse)
    else:
        ws = csa2.workspace(csa2.paged_attn_workspace_size(B, n, 0))
        csa2.paged_attn_decode(planes, pages, B, counts, n, None, 0, q, SCALE, out, ws, lse_out=lse)
    assert csa2.check(ws)[0] == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("at", [0, 63, 40_001, 65_535])
def test_rows_far_behind_one_add_up(prefix, at):
    """Row `at` is 1 in channels 0 .. 255 and 0 in the others, all other rows the opposite, and head h's query a_h
    and 0: the others' logits are 0, the strong row's z = 256 a_h / sqrt(512), from 6 to 20 nats above them.
    152 queries, so that a CTA (or pair) runs all rows of one.

    With w = e^-z: out = 1 / (1 + (n - 1) w) in the first half and (n - 1) w / (1 + (n - 1) w) in the second.
    Errors of the second half: each w is rounded to f16 (2^-11), and again with the sum (2^-11), moves by the
    logit's error e_z = z 2^-16 + 2^-20 in numerator and denominator, fp32 sums add 2^-14, and of a weight at
    most 2^-36 of the strongest row's is lost."""
    n, P, B = 65_536, 64, 152
    codes = np.zeros((n, 256), np.uint8)
    codes[:, 128:] = 0x22  # E2M1 code 2 is 1.0
    codes[at] = codes[at, ::-1]
    a = torch.linspace(0.5, 1.8, H).to(torch.bfloat16)
    q = torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, :256] = a.cuda()[None, :, None]
    out, lse = attend(prefix, codes, np.full((n, 32), 0x38, np.uint8), n, P, q, B)
    z = a.double().numpy() * 256 * SCALE
    w = np.exp(-z)
    den = 1 + (n - 1) * w
    ez = z * 2.0 ** -16 + 2.0 ** -20
    rel = 2 * 2.0 ** -11 + 2 * ez + 2.0 ** -14
    lost = (n - 1) * np.minimum(w, 2.0 ** -36) / den
    for half, want in ((out[..., :256], 1 / den), (out[..., 256:], (n - 1) * w / den)):
        err = np.abs(half - want[None, :, None]).max((0, 2))
        assert (err <= want * rel + lost).all(), (err / (want * rel + lost)).max()
    assert (np.abs(lse - (z + np.log(den))) <= ez + 2.0 ** -14).all()
