"""Refusals of the binding's draft-tree, append and rotation calls, before the library is asked (no GPU needed)."""
import pytest

import compressed_sparse_attention_nvfp4_gb300 as csa2

torch = pytest.importorskip("torch")
PLANES, PAGES, TREES = csa2.Planes(256, 256, 256, 256, 64), csa2.Pages(16, 8, 32), csa2.Trees(16, 16, 4, 20, 8, 1)
WS = torch.empty(16, dtype=torch.uint8)  # too small: status 3 for a call that is right otherwise
I32, I64 = torch.int32, torch.int64


def status(call):
    with pytest.raises(csa2.Csa2Error) as e:
        call()
    return e.value.status


def attn(**kw):
    a = dict(n_entries=16, swa_pos=16, q_pos=16) | kw
    return status(lambda: csa2.tree_attn_decode(PLANES, PAGES, TREES, a["n_entries"], 100, 256, a["swa_pos"], 256, 128, 256,
                                                a["q_pos"], 0.04, 256, WS, out_type=csa2.OUT_BF16))


def commit(**kw):
    a = dict(n_entries=16, n_accept=16, path=16, n_new=16, pos=16, ring_pos=16) | kw
    return status(lambda: csa2.tree_commit(PLANES, PAGES, TREES, a["n_entries"], a["n_accept"], a["path"], 8, a["n_new"], WS,
                                           draft=256, pos=a["pos"], ring=256, ring_pos=a["ring_pos"], n_win=128))


def append(**kw):
    a = dict(slot=16, entry=16, pos=16) | kw
    return status(lambda: csa2.latent_append(torch.empty(4, 512), 4, PLANES, 8, a["slot"], a["entry"], WS, pos=a["pos"]))


SHAPES = {"n_entries": (4,), "n_accept": (4,), "path": (4, 8), "n_new": (4,), "swa_pos": (4, 128), "ring_pos": (4, 128),
          "q_pos": (20,), "slot": (4,), "entry": (4,)}
INTS = [(attn, "n_entries", I32), (attn, "swa_pos", I64), (attn, "q_pos", I64), (commit, "n_entries", I32),
        (commit, "n_accept", I32), (commit, "path", I32), (commit, "n_new", I32), (commit, "pos", I64),
        (commit, "ring_pos", I64), (append, "slot", I32), (append, "entry", I64), (append, "pos", I64)]


@pytest.mark.parametrize("call,name,dtype", INTS)
def test_index_tensors_are_of_the_type_that_is_read(call, name, dtype):
    shape = SHAPES.get(name, (4,))
    t = torch.zeros(shape, dtype=dtype)
    assert call(**{name: t}) == 3 and call(**{name: 16}) == 3
    wide = torch.zeros((*shape[:-1], 2 * shape[-1]), dtype=dtype)
    for bad in (t.to(I64 if dtype == I32 else I32), t.to(torch.int16), t.float(), wide[..., ::2]):
        assert call(**{name: bad}) == 1


def test_trees_are_int32():
    start, parent = torch.zeros(5, dtype=I32), torch.zeros(20, dtype=I32)
    assert csa2.trees(start, parent, 4, 20, 8).start == start.data_ptr()
    assert csa2.trees(start, None, 4, 20, 8).parent is None and csa2.trees(16, 32, 4, 20, 8).parent == 32
    for a, b in ((start.long(), parent), (start, parent.long()), (torch.zeros(10, dtype=I32)[::2], parent), (start, parent.float())):
        assert status(lambda: csa2.trees(a, b, 4, 20, 8)) == 1


def test_rope_positions_are_int64():
    x, rot = torch.empty(4, 8, 128), csa2.rotary(64)
    csa2.rope(x, 0, 8, 128, torch.zeros(4, dtype=I64), rot, x)
    for bad in (torch.zeros(4, dtype=I32), torch.zeros(4), torch.zeros(8, dtype=I64)[::2]):
        assert status(lambda: csa2.rope(x, 0, 8, 128, bad, rot, x)) == 1


def test_rope_tensors_have_the_rows_that_are_asked_for():
    x, few, pos, rot = torch.empty(4, 8, 128), torch.empty(3, 8, 128), torch.zeros(4, dtype=I64), csa2.rotary(64)
    rope = lambda a, b, n: csa2.rope(a, n, 8, 128, pos, rot, b)  # noqa: E731
    rope(x, x, 0)  # more rows than are turned
    for a, b in ((few, x), (x, few), (few.view(3, 1024), x), (torch.empty(0, 8, 128), x)):
        assert status(lambda: rope(a, b, 4)) == 1


def test_append_takes_rows_of_latents_and_keys():
    E = torch.empty
    f = lambda x, key: status(lambda: csa2.latent_append(x, 4, PLANES, 8, 16, 16, WS, key=key))  # noqa: E731
    for x, key in ((E(4, 512), E(4, 128)), (E(9, 512), E(2, 2, 128)), (E(2048), E(513)), (None, E(4, 128)), (E(4, 512), None)):
        assert f(x, key) == 3  # right but for the workspace
    for x, key in ((E(3, 512), None), (E(4, 256), None), (E(4, 1024), None), (E(2047), None), (E(0, 512), None),
                   (None, E(3, 128)), (None, E(4, 512)), (None, E(4, 64)), (E(4, 512), E(4, 127))):
        assert f(x, key) == 1
