"""Host-side checks of the paged-cache entry points: every refusal comes back before a launch (no GPU
needed; the pointers are aligned numbers that nothing reads), and the workspace queries."""
import ctypes

import pytest

import compressed_sparse_attention_nvfp4_gb300 as csa2

FAKE = csa2.KVPlanes(256, 256, 256, 256, 64)


def tables(B=4, have=16, new=16, page=64, m=1, kept=None, table=16, max_pages=8, n_pages=32, free=16, n_free=16,
           n_free_out=16, n_entries=16, n_rows=0, query=None, slot=None, entry=None, pos=None, start=None, ws=256,
           ws_bytes=1 << 20):
    return csa2.lib().csa2_page_tables(B, have, new, page, m, kept, table, max_pages, n_pages, free, n_free,
                                       n_free_out, n_entries, n_rows, query, slot, entry, pos, start, ws, ws_bytes,
                                       None)


@pytest.mark.parametrize("bad", [dict(B=0), dict(B=65536), dict(have=None), dict(new=None), dict(page=0),
                                 dict(page=-1), dict(m=0), dict(table=None), dict(max_pages=-1), dict(n_pages=0),
                                 dict(free=None), dict(n_free=None), dict(n_free_out=None), dict(n_entries=None),
                                 dict(n_rows=-1), dict(n_rows=5), dict(have=18), dict(kept=2), dict(table=6),
                                 dict(entry=12, n_rows=1), dict(pos=20, n_rows=1), dict(slot=3, n_rows=1),
                                 dict(start=9)])
def test_page_tables_refuses(bad):
    assert tables(**bad) == 1


def test_page_tables_workspace():
    need = csa2.page_tables_workspace_size(4)
    assert need > 0 and need % 256 == 0
    assert tables(ws=None) == 3
    assert tables(ws=128) == 3
    assert tables(ws_bytes=need - 1) == 3
    assert csa2.page_tables_workspace_size(0) == 0
    assert csa2.page_tables_workspace_size(65535) >= 4 * 4 * 65535


def attn(prefix, planes=FAKE, pages=(16, 8, 32), B=4, n=16, n_max=100, swa=16, n_swa=128, q=16, scale=0.04, nr=None,
         q_pos=None, sink=None, win=None, out=16, out_type=1, lse=None, ws=256, ws_bytes=1 << 40, G=2, start=16,
         shared=16, shared_max=100, own_max=20):
    L = csa2.lib()
    pg = None if pages is None else ctypes.byref(csa2.Pages(*pages))
    tail = (swa, n_swa, q, scale, nr, q_pos, sink, win, out, out_type, lse, ws, ws_bytes, None)
    if prefix:
        return L.csa2_prefix_attn_decode(ctypes.byref(planes), pg, B, n, G, start, shared, shared_max, own_max, *tail)
    return L.csa2_paged_attn_decode(ctypes.byref(planes), pg, B, n, n_max, *tail)


COMMON = [dict(planes=csa2.KVPlanes(None, 16, 16, 16, 64)), dict(planes=csa2.KVPlanes(256, 256, 256, 256, 0)),
          dict(planes=csa2.KVPlanes(8, 256, 256, 256, 64)), dict(planes=csa2.KVPlanes(256, 256, 256, 256, 1 << 31)),
          dict(pages=None), dict(pages=(None, 8, 32)), dict(pages=(18, 8, 32)), dict(pages=(16, -1, 32)),
          dict(pages=(16, 8, -1)), dict(pages=(16, 1, 32)), dict(B=0), dict(B=65536), dict(n=None), dict(n=18),
          dict(swa=None), dict(swa=24), dict(n_swa=-1), dict(n_swa=129), dict(q=None), dict(q=8), dict(scale=0.0),
          dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(out=8),
          dict(out_type=2), dict(out_type=-1), dict(sink=18), dict(q_pos=12)]


@pytest.mark.parametrize("bad", COMMON + [dict(n_max=-1), dict(n_max=65537), dict(n_max=513)])
def test_paged_attn_refuses(bad):
    assert attn(False, **bad) == 1


@pytest.mark.parametrize("bad", COMMON + [dict(G=0), dict(G=5), dict(start=None), dict(start=18), dict(shared=None),
                                          dict(shared=6), dict(shared_max=-1), dict(own_max=-1), dict(own_max=513),
                                          dict(shared_max=513),
                                          dict(pages=(16, 1 << 20, 32), shared_max=65537),
                                          dict(pages=(16, 1 << 20, 32), own_max=65537)])
def test_prefix_attn_refuses(bad):
    assert attn(True, **bad) == 1


@pytest.mark.parametrize("prefix", [False, True])
def test_attn_norm_rope_and_window_arguments(prefix):
    for bad in (csa2.NormRope(None, 1e-6, 1, 1.0), csa2.NormRope(None, -1.0, 0, 10000.0),
                csa2.NormRope(4, 1e-6, 0, 10000.0)):
        assert attn(prefix, nr=ctypes.byref(bad), q_pos=16) == 1
    assert attn(prefix, nr=ctypes.byref(csa2.NormRope(None, 1e-6, 1, 10000.0))) == 1  # rotation without positions
    for bad in (csa2.Window(None, 16), csa2.Window(16, None), csa2.Window(12, 16)):
        assert attn(prefix, win=ctypes.byref(bad)) == 1


@pytest.mark.parametrize("prefix", [False, True])
def test_attn_workspace(prefix):
    need = csa2.prefix_attn_workspace_size(4, 2, 100, 20, 128) if prefix else csa2.paged_attn_workspace_size(4, 100, 128)
    assert need > 0
    assert attn(prefix, ws=None) == 3
    assert attn(prefix, ws=128) == 3
    assert attn(prefix, ws_bytes=need - 1) == 3


def test_workspace_queries_of_refused_sizes():
    assert csa2.paged_attn_workspace_size(0, 100, 128) == 0
    assert csa2.paged_attn_workspace_size(1, 65537, 128) == 0
    assert csa2.prefix_attn_workspace_size(4, 5, 100, 20, 128) == 0
    assert csa2.prefix_attn_workspace_size(4, 1, 65537, 600, 128) == 0
    assert csa2.prefix_attn_workspace_size(4, 1, -1, 20, 128) == 0


def test_out_type_follows_the_tensor():
    class T:
        def __init__(self, dtype):
            self.dtype = dtype
    assert csa2._out_type(T("torch.bfloat16"), None) == csa2.OUT_BF16
    assert csa2._out_type(T("torch.float32"), None) == csa2.OUT_F32
    assert csa2._out_type(12345, None) == csa2.OUT_F32
    with pytest.raises(csa2.Csa2Error):
        csa2._out_type(T("torch.float16"), None)


def test_status_string_of_missing_pages():
    assert csa2.status_string(7) and csa2.STATUS[7] == "CSA2_ERR_NO_PAGES"
