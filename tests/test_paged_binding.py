"""Refusals of the binding's paged attention calls, before the library is asked (no GPU needed)."""
import pytest

import compressed_sparse_attention_nvfp4_gb300 as csa2

torch = pytest.importorskip("torch")
PLANES, PAGES = csa2.Planes(256, 256, 256, 256, 64), csa2.Pages(16, 8, 32)


def status(call, **kw):
    ws = torch.empty(16, dtype=torch.uint8)  # too small: status 3 for a call that is right otherwise
    with pytest.raises(csa2.Csa2Error) as e:
        if call == "paged":
            csa2.paged_attn_decode(PLANES, PAGES, 4, 16, 100, 16, 128, 16, 0.04, ws=ws, **kw)
        else:
            csa2.prefix_attn_decode(PLANES, PAGES, 4, 16, 2, 16, 16, 100, 20, 16, 128, 16, 0.04, ws=ws, **kw)
    return e.value.status


@pytest.mark.parametrize("call", ["paged", "prefix"])
def test_the_output_type_has_to_be_known(call):
    assert status(call, out=256) == 1
    assert status(call, out=256, out_type=csa2.OUT_BF16) == 3
    assert status(call, out=256, out_type=csa2.OUT_F32) == 3
    f32, bf16 = torch.empty(16), torch.empty(16, dtype=torch.bfloat16)
    assert status(call, out=f32) == 3 and status(call, out=f32, out_type=csa2.OUT_F32) == 3
    assert status(call, out=bf16) == 3 and status(call, out=bf16, out_type=csa2.OUT_BF16) == 3
    assert status(call, out=f32, out_type=csa2.OUT_BF16) == 1
    assert status(call, out=bf16, out_type=csa2.OUT_F32) == 1
    assert status(call, out=torch.empty(16, dtype=torch.float16)) == 1


def test_a_page_table_is_contiguous_int32():
    t = torch.zeros((4, 16), dtype=torch.int32)
    assert csa2.pages(t, 32).max_pages == 16 and csa2.pages(t[1:3], 32).max_pages == 16
    assert csa2.pages(256, 32, max_pages=8).max_pages == 8
    for bad in (t[:, :8], t.t(), t.long(), t.to(torch.int16)):
        with pytest.raises(csa2.Csa2Error) as e:
            csa2.pages(bad, 32)
        assert e.value.status == 1
