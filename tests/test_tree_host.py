"""Host-side checks of the rotary, latent-append and draft-tree entry points: every refusal comes back before a
launch (no GPU needed; the pointers are aligned numbers that nothing reads), the binding's own refusals, and the
workspace queries."""
import ctypes

import pytest

import compressed_sparse_attention_nvfp4_gb300 as csa2

torch = pytest.importorskip("torch")
FAKE = csa2.KVPlanes(256, 256, 256, 256, 64)
ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
NAN, INF = float("nan"), float("inf")

BAD_SCALINGS = [csa2.rope_scaling(3, 2.0), csa2.rope_scaling(-1, 2.0), csa2.rope_scaling(1, 0.0), csa2.rope_scaling(1, -2.0),
                csa2.rope_scaling(1, NAN), csa2.rope_scaling(1, INF), csa2.rope_scaling(2, 4.0, 0),
                csa2.rope_scaling(2, 4.0, 4096, 1.0, 1.0), csa2.rope_scaling(2, 4.0, 4096, 32.0, 0.0),
                csa2.rope_scaling(2, 4.0, 4096, NAN, 1.0), csa2.rope_scaling(2, 4.0, 4096, INF, 1.0),
                csa2.rope_scaling(2, 0.0, 4096)]
BAD_ROTARIES = [csa2.rotary(64, layout=2), csa2.rotary(64, layout=-1), csa2.rotary(0), csa2.rotary(63), csa2.rotary(-2),
                csa2.rotary(514), csa2.rotary(64, -1), csa2.rotary(64, 65), csa2.rotary(64, base=1.0),
                csa2.rotary(64, base=NAN), csa2.rotary(64, base=INF), csa2.rotary(64, magnitude=NAN),
                csa2.rotary(64, magnitude=INF)] + [csa2.rotary(64, scaling=s) for s in BAD_SCALINGS]


def rope(x=256, x_row=1024, x_head=128, y=512, y_row=1024, y_head=128, type=1, rows=4, heads=8, dim=128, pos=16,
         rot=csa2.rotary(64)):
    return csa2.lib().csa2_rope(x, x_row, x_head, y, y_row, y_head, type, rows, heads, dim, pos, ref(rot), 0, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(y=None), dict(pos=None), dict(rot=None), dict(type=2), dict(type=-1),
                                 dict(rows=-1), dict(rows=1 << 31), dict(heads=0), dict(heads=65536), dict(dim=0),
                                 dict(dim=65537), dict(dim=63), dict(x=257), dict(y=515), dict(pos=12), dict(x=258, type=0),
                                 dict(y_head=127), dict(y_row=1023), dict(y_row=-1024), dict(y_head=0),
                                 dict(y=256, y_row=2048), dict(y=256, x_head=256, x_row=2048, y_row=2048),
                                 dict(x_row=1 << 40), dict(y_row=1 << 40), dict(x_head=1 << 62)]
                         + [dict(rot=r) for r in BAD_ROTARIES])
def test_rope_refuses(bad):
    assert rope(**bad) == 1


def test_rope_of_no_rows():
    assert rope(rows=0, x=None, y=None, pos=None) == 0


def append(x=256, key=256, type=0, R=4, planes=FAKE, n_slots=8, slot=16, entry=16, nr=csa2.norm_rope(256, 1e-6, True),
           scaling=None, pos=16, key_rot=csa2.rotary(64), ws=256, ws_bytes=256):
    return csa2.lib().csa2_latent_append(x, key, type, R, ref(planes), n_slots, slot, entry, ref(nr), ref(scaling), pos,
                                         ref(key_rot), ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(x=264), dict(key=264), dict(type=2), dict(R=-1), dict(R=(1 << 30) + 1),
                                 dict(planes=csa2.KVPlanes(256, 256, 256, 256, 0)), dict(planes=csa2.KVPlanes(8, 256, 256, 256, 4)),
                                 dict(n_slots=0), dict(slot=None), dict(entry=None), dict(slot=18), dict(entry=20), dict(pos=None),
                                 dict(pos=None, key_rot=None), dict(pos=None, nr=None), dict(pos=20),
                                 dict(nr=csa2.norm_rope(8, 1e-6)), dict(nr=csa2.norm_rope(256, -1.0)),
                                 dict(nr=csa2.norm_rope(256, 1e-6, True, 1.0)), dict(key_rot=csa2.rotary(130)),
                                 dict(key_rot=csa2.rotary(64, 65))]
                         + [dict(scaling=s) for s in BAD_SCALINGS] + [dict(key_rot=r) for r in BAD_ROTARIES])
def test_latent_append_refuses(bad):
    assert append(**bad) == 1


def test_latent_append_workspace():
    assert csa2.latent_append_workspace_size(5) == 256 and csa2.latent_append_workspace_size(-1) == 0
    assert append(ws=None) == 3 and append(ws=128) == 3 and append(ws_bytes=255) == 3


def commit(kv=FAKE, pages=csa2.Pages(16, 8, 32), trees=csa2.Trees(16, None, 4, 20, 8, 1), n=16, accept=16, path=16, n_path=8,
           new=16, draft=256, pos=16, ring=256, ring_pos=16, n_win=128, ws=256, ws_bytes=256):
    return csa2.lib().csa2_tree_commit(ref(kv), ref(pages), ref(trees), n, accept, path, n_path, new, draft, pos, ring,
                                       ring_pos, n_win, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(kv=None), dict(kv=csa2.KVPlanes(256, 256, 256, 256, 0)), dict(pages=None),
                                 dict(kv=csa2.KVPlanes(256, 256, 256, 256, 1 << 31)),
                                 dict(pages=csa2.Pages(None, 8, 32)), dict(pages=csa2.Pages(18, 8, 32)),
                                 dict(pages=csa2.Pages(16, -1, 32)), dict(pages=csa2.Pages(16, 8, -1)), dict(trees=None),
                                 dict(trees=csa2.Trees(None, None, 4, 20, 8, 1)), dict(trees=csa2.Trees(18, None, 4, 20, 8, 1)),
                                 dict(trees=csa2.Trees(16, None, 0, 20, 8, 1)), dict(trees=csa2.Trees(16, None, 65536, 20, 8, 1)),
                                 dict(trees=csa2.Trees(16, None, 4, -1, 8, 1)), dict(trees=csa2.Trees(16, None, 4, 20, 0, 1)),
                                 dict(trees=csa2.Trees(16, None, 4, 20, 65, 1)), dict(n=None), dict(n=18), dict(accept=None),
                                 dict(accept=18), dict(path=None), dict(path=18), dict(n_path=-1), dict(new=18), dict(n_win=-1),
                                 dict(draft=None), dict(draft=264), dict(pos=None), dict(pos=20), dict(ring=None), dict(ring=264),
                                 dict(ring_pos=None), dict(ring_pos=20)])
def test_tree_commit_refuses(bad):
    assert commit(**bad) == 1


def test_tree_commit_workspace():
    assert csa2.tree_commit_workspace_size(5) == 256
    assert csa2.tree_commit_workspace_size(0) == 0 and csa2.tree_commit_workspace_size(65536) == 0
    assert commit(ws=None) == 3 and commit(ws=128) == 3 and commit(ws_bytes=255) == 3
    off = csa2.Trees(16, None, 4, 20, 8, 0)
    assert commit(kv=None, pages=None, n=None, trees=off, ws=None) == 3  # without entries no cache is needed
    assert commit(draft=None, pos=None, ring=None, ring_pos=None, n_win=0, ws=None) == 3


TREES = csa2.Trees(16, 16, 4, 20, 8, 1)


def attn(kv=FAKE, pages=csa2.Pages(16, 8, 32), trees=TREES, n=16, n_max=100, swa=256, swa_pos=16, draft=256, n_swa=128, q=256,
         q_pos=16, scale=0.04, nr=None, scaling=None, sink=None, out=256, out_type=1, lse=None, ws=256, ws_bytes=1 << 40):
    return csa2.lib().csa2_tree_attn_decode(ref(kv), ref(pages), ref(trees), n, n_max, swa, swa_pos, draft, n_swa, q, q_pos, scale,
                                            ref(nr), ref(scaling), sink, out, out_type, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(kv=None), dict(kv=csa2.KVPlanes(None, 256, 256, 256, 64)),
                                 dict(kv=csa2.KVPlanes(256, 256, 256, 256, 0)), dict(kv=csa2.KVPlanes(256, 256, 256, 256, 1 << 31)),
                                 dict(pages=None), dict(pages=csa2.Pages(None, 8, 32)), dict(pages=csa2.Pages(18, 8, 32)),
                                 dict(pages=csa2.Pages(16, -1, 32)), dict(pages=csa2.Pages(16, 8, -1)),
                                 dict(pages=csa2.Pages(16, 1, 32)), dict(pages=csa2.Pages(16, 8, 1 << 25)),
                                 dict(n_max=505), dict(n_max=512, trees=csa2.Trees(16, 16, 4, 20, 1, 1)), dict(trees=None),
                                 dict(trees=csa2.Trees(None, 16, 4, 20, 8, 1)), dict(trees=csa2.Trees(16, None, 4, 20, 8, 1)),
                                 dict(trees=csa2.Trees(18, 16, 4, 20, 8, 1)), dict(trees=csa2.Trees(16, 18, 4, 20, 8, 1)),
                                 dict(trees=csa2.Trees(16, 16, 0, 20, 8, 1)), dict(trees=csa2.Trees(16, 16, 65536, 20, 8, 1)),
                                 dict(trees=csa2.Trees(16, 16, 4, 0, 8, 1)), dict(trees=csa2.Trees(16, 16, 4, 65536, 8, 1)),
                                 dict(trees=csa2.Trees(16, 16, 4, 20, 0, 1)), dict(trees=csa2.Trees(16, 16, 4, 20, 65, 1)),
                                 dict(n=None), dict(n=18), dict(n_max=-1), dict(n_max=65537), dict(n_swa=-1), dict(n_swa=129),
                                 dict(swa=None), dict(swa=264), dict(swa_pos=None), dict(swa_pos=20), dict(draft=None),
                                 dict(draft=264), dict(q=None), dict(q=264), dict(q_pos=None), dict(q_pos=20), dict(scale=0.0),
                                 dict(scale=NAN), dict(scale=INF), dict(nr=csa2.norm_rope(8, 1e-6)),
                                 dict(nr=csa2.norm_rope(None, 1e-6, True), q_pos=None, n_swa=0), dict(sink=18), dict(out=None),
                                 dict(out=264), dict(out_type=2), dict(lse=18)] + [dict(scaling=s) for s in BAD_SCALINGS])
def test_tree_attn_refuses(bad):
    assert attn(**bad) == 1


def test_tree_attn_workspace():
    need = csa2.tree_attn_workspace_size(4, 20, 8, 100, 128)
    assert need > 0 and need % 256 == 0
    assert attn(ws=None) == 3 and attn(ws=128) == 3 and attn(ws_bytes=need - 1) == 3
    # right for a window that is not there, a table that just holds the bound, drafts without entries
    assert attn(swa=None, swa_pos=None, draft=None, q_pos=None, n_swa=0, ws=None) == 3
    assert attn(n_max=504, ws=None) == 3 and attn(n_max=512, trees=csa2.Trees(16, 16, 4, 20, 8, 0), ws=None) == 3
    for bad in ((0, 20, 8, 100, 128), (4, 0, 8, 100, 128), (65536, 20, 8, 100, 128), (4, 65536, 8, 100, 128), (4, 20, 0, 100, 128),
                (4, 20, 65, 100, 128), (4, 20, 8, -1, 128), (4, 20, 8, 65537, 128), (4, 20, 8, 100, -1)):
        assert csa2.tree_attn_workspace_size(*bad) == 0


def refused(call):
    with pytest.raises(csa2.Csa2Error) as e:
        call()
    return e.value.status


def test_binding_of_rope_wants_one_type_and_strides_that_fit():
    pos, rot, E = torch.zeros(4, dtype=torch.int64), csa2.rotary(64), torch.empty
    f = lambda x, out, **kw: refused(lambda: csa2.rope(x, 4, 8, 128, pos, rot, out, **kw))  # noqa: E731
    x, h = E(4, 8, 128), E(4, 8, 128, dtype=torch.bfloat16)
    assert f(x, h) == 1 and f(h, x) == 1 and f(x, x, type=csa2.BF16) == 1 and f(256, 512) == 1 and f(x.half(), x.half()) == 1
    assert f(E(4, 8, 64), x) == 1 and f(x, E(4, 7, 128)) == 1 and f(E(4, 128, 8).transpose(1, 2), x) == 1


def test_binding_of_latent_append_wants_one_type_and_dense_rows():
    planes, ws = csa2.Planes(256, 256, 256, 256, 64), torch.empty(16, dtype=torch.uint8)
    f = lambda x, key=None, **kw: refused(lambda: csa2.latent_append(x, 4, planes, 8, 16, 16, ws, key=key, **kw))  # noqa: E731
    x, key = torch.empty(4, 512), torch.empty(4, 128)
    assert f(x, key) == 3  # right but for the workspace
    assert f(x, key.bfloat16()) == 1 and f(x.half()) == 1 and f(x, type=csa2.BF16) == 1 and f(256) == 1
    assert f(256, type=csa2.F32) == 3 and f(torch.empty(4, 1024)[:, :512]) == 1 and f(None, key) == 3
