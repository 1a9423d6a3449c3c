"""Host-side checks of the entry points for drafted trees and windows: sizes and refusals (every
argument is checked before any CUDA call, so they need no GPU), and the tests' own restatement on
hand-worked trees."""
import ctypes

import numpy as np
import pytest

import kv_tree_reference as tree_ref
import moe_expert_offload_gb300 as m
from test_kv_cpu import BATCH, POOL, PTR, SHAPES, TABLES, _batch, _kv, _refused


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_expert_offload_gb300 import _build

    _build.build()


def _tree(**kw):
    f = dict(max_new=8, parent=PTR, seen=PTR)
    f.update(kw)
    return m.MoeKvTree(**f)


def _view(window=0, sinks=0, tree=None):
    return m.MoeKvView(window, sinks, ctypes.pointer(tree) if tree is not None else None)


def _plan(batch=None, view=None, rows=4, T=16):
    return m.moe_kv_tree_plan(batch or _batch(), view or _view(tree=_tree()), rows, T, 0)


def _attend(kv=None, batch=None, view=None, rows=4, q=PTR, T=16, heads=8, max_new=4, scale=0.1,
            ws=PTR, n=1 << 40, out=PTR):
    return m.moe_kv_attention_view(kv or _kv(), batch or _batch(), view or _view(16, 4, _tree()),
                                   rows, q, T, heads, max_new, scale, ws, n, out, 0)


def _accept(batch=None, tree=None, rows=4, T=16, **kw):
    a = dict(token=PTR, next_token=PTR, path=PTR, kept=PTR, drop=PTR, last=PTR)
    a.update(kw)
    return m.moe_kv_tree_accept(batch or _batch(), tree or _tree(), rows, T, stream=0, **a)


def _keep(layers=None, batch=None, rows=4, T=16, path=PTR, kept=PTR):
    return m.moe_kv_tree_keep(layers or [_kv(), _kv()], batch or _batch(), rows, T, path, kept, 0)


def test_words():
    for n in (1, 31, 32, 33, 64, 65, 255, 256):
        assert m.moe_kv_tree_words(n) == 1 + -(-n // 32)
    for n in (0, -1, 257, 2 ** 31 - 1, -2 ** 31):
        assert m.moe_kv_tree_words(n) == 0


@pytest.mark.parametrize("kw,code", SHAPES)
def test_shape_refusals(kw, code):
    _refused(code, lambda: _attend(_kv(**kw)))
    _refused(code, lambda: _keep([_kv(**kw)]))


@pytest.mark.parametrize("kw,code", TABLES)
def test_table_refusals(kw, code):
    _refused(code, lambda: _attend(_kv(**kw)))


@pytest.mark.parametrize("kw,code", POOL)
def test_pool_refusals(kw, code):
    _refused(code, lambda: _attend(_kv(**kw)), "pool")
    for layers in ([_kv(**kw)], [_kv(), _kv(**kw)]):
        _refused(code, lambda: _keep(layers), "pool")


@pytest.mark.parametrize("kw,code", BATCH)
def test_batch_refusals(kw, code):
    b = _batch(**kw)
    for call in (lambda: _plan(batch=b, rows=1, T=1), lambda: _attend(batch=b, rows=1, T=1),
                 lambda: _accept(batch=b, rows=1, T=1), lambda: _keep(batch=b, rows=1, T=1)):
        _refused(code, call)


def test_rows_and_tokens():
    for call in (_plan, _attend, _accept, _keep):
        for rows, code in ((0, m.MOE_EINVAL), (-1, m.MOE_EINVAL), (5, m.MOE_ECAPACITY)):
            _refused(code, lambda: call(rows=rows), "rows")
        for T, code in ((-1, m.MOE_EINVAL), (17, m.MOE_ECAPACITY)):
            _refused(code, lambda: call(T=T), "T")
    # nothing to do launches nothing
    assert _plan(T=0) == m.MOE_OK and _attend(T=0) == m.MOE_OK and _keep(T=0) == m.MOE_OK


def test_view_refusals():
    for kw, words in ((dict(window=-1), "window"), (dict(sinks=-1, window=3), "sinks"),
                      (dict(window=-2 ** 31), "window"), (dict(tree=_tree(max_new=0)), "max_new"),
                      (dict(tree=_tree(max_new=257)), "max_new"), (dict(tree=_tree(max_new=-1)), "max_new"),
                      (dict(tree=_tree(parent=None)), "parent"), (dict(tree=_tree(seen=None)), "seen")):
        _refused(m.MOE_EINVAL, lambda: _attend(view=_view(**kw)), words)
        if "tree" not in kw:
            kw["tree"] = _tree()
        _refused(m.MOE_EINVAL, lambda: _plan(view=_view(**kw)), words)
    _refused(m.MOE_EINVAL, lambda: _plan(view=_view(5, 1)), "tree")
    # a visibility of more than 2^31 - 1 words
    big = _batch(max_tokens=2 ** 31 - 1)
    wide = _view(tree=_tree(max_new=256))
    _refused(m.MOE_EUNSUPPORTED, lambda: _plan(batch=big, view=wide, T=240_000_000), "words")
    _refused(m.MOE_EUNSUPPORTED, lambda: _attend(batch=big, view=wide, T=240_000_000), "words")
    L = m.lib()
    kv, b = _kv(), _batch()
    assert L.moe_kv_attention_view(kv, b, None, 4, PTR, 16, 8, 4, 0.1, PTR, 1 << 40, PTR, 0) == m.MOE_EINVAL
    assert L.moe_kv_tree_plan(b, None, 4, 16, 0) == m.MOE_EINVAL
    assert L.moe_kv_tree_accept(b, None, 4, 16, PTR, PTR, PTR, PTR, PTR, PTR, 0) == m.MOE_EINVAL
    assert L.moe_kv_tree_keep(None, 2, b, 4, 16, PTR, PTR, 0) == m.MOE_EINVAL
    assert L.moe_kv_tree_keep(kv, 0, b, 4, 16, PTR, PTR, 0) == m.MOE_EINVAL


@pytest.mark.parametrize("kw,words", [
    (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(q=PTR + 8), "alignment"), (dict(out=PTR + 2), "alignment"), (dict(ws=PTR + 128), "alignment"),
    (dict(scale=0.0), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(scale=-1.0), "scale"), (dict(heads=7), "heads"), (dict(heads=0), "heads"),
    (dict(max_new=0), "max_new"),
])
def test_attention_refusals(kw, words):
    _refused(m.MOE_EINVAL, lambda: _attend(**kw), words)


def test_attention_workspace():
    need = m.moe_kv_attention_workspace_bytes(_kv(), 4, 16, 8, 4)
    _refused(m.MOE_ECAPACITY, lambda: _attend(n=need - 1), "workspace")
    _refused(m.MOE_EUNSUPPORTED, lambda: _attend(heads=130), "query heads")


def test_accept_and_keep_refusals():
    for name in ("token", "next_token", "path", "kept", "drop", "last"):
        _refused(m.MOE_EINVAL, lambda: _accept(**{name: None}), "NULL")
    for kw in (dict(max_new=0), dict(max_new=257), dict(parent=None)):
        _refused(m.MOE_EINVAL, lambda: _accept(tree=_tree(**kw)), "tree")
    _refused(m.MOE_EINVAL, lambda: _keep(path=None), "NULL")
    _refused(m.MOE_EINVAL, lambda: _keep(kept=None), "NULL")
    for kw in (dict(num_blocks=9), dict(block_tokens=32), dict(kv_heads=3), dict(head_dim=64)):
        _refused(m.MOE_EINVAL, lambda: _keep([_kv(), _kv(), _kv(**kw)]), "layer 2")


def test_binding_refuses_arrays_that_do_not_fit():
    torch = pytest.importorskip("torch")
    good, short = torch.zeros(16, dtype=torch.int32), torch.zeros(15, dtype=torch.int32)
    wide, gaps = torch.zeros(16, dtype=torch.int64), torch.zeros(32, dtype=torch.int32)[::2]
    for bad in (short, wide, gaps):
        for name in ("token", "next_token", "path"):
            _refused(m.MOE_EINVAL, lambda: _accept(**{name: bad}), name)
        _refused(m.MOE_EINVAL, lambda: _keep(path=bad), "path")
    for bad in (torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)):
        for name in ("kept", "drop", "last"):
            _refused(m.MOE_EINVAL, lambda: _accept(**{name: bad}), name)
        _refused(m.MOE_EINVAL, lambda: _keep(kept=bad), "kept")
    for bad in (torch.zeros(16 * 8 * 128, dtype=torch.float16), torch.zeros(9, dtype=torch.bfloat16)):
        _refused(m.MOE_EINVAL, lambda: _attend(q=bad), "q")
        _refused(m.MOE_EINVAL, lambda: _attend(out=bad), "out")
    tree = m.DeviceKvTree(15, 4, 8, device="cpu")
    assert tuple(tree.seen.shape) == (15, 2)
    view = m.make_view(16, 4, tree)
    _refused(m.MOE_EINVAL, lambda: _plan(view=view), "15")
    _refused(m.MOE_EINVAL, lambda: _attend(view=view), "15")
    _refused(m.MOE_EINVAL, lambda: _accept(tree=tree.c), "15")
    for n in (0, 257):
        _refused(m.MOE_EINVAL, lambda: m.DeviceKvTree(16, 4, n, device="cpu"), "max_new")
    _refused(m.MOE_EINVAL, lambda: m.DeviceKvTree(16, 4, 8, device="cpu", parent=short), "parent")
    other = m.DeviceKvTree(16, 4, 8, device="cpu", parent=good)
    assert other.c.parent == good.data_ptr()


def test_the_restatement_on_worked_trees():
    #        0
    #      1   2        3 (follows the cached tokens)
    #    4   5           \
    #        6            7
    parents = [-1, 0, 0, -1, 1, 1, 5, 3]
    depth, path = tree_ref.depths_and_paths(parents)
    assert depth == [0, 1, 1, 0, 2, 2, 3, 1] and depth == tree_ref.depths(parents)
    assert path[6] == [0, 1, 5, 6] and path[7] == [3, 7]
    see = tree_ref.own_visible(parents, 100, 3, 0)
    assert np.flatnonzero(see[6]).tolist() == [1, 5, 6] and np.flatnonzero(see[4]).tolist() == [0, 1, 4]
    # positions 1 .. 4 with one cached token: a sink at 0 .. 1 keeps token 0 in sight
    see = tree_ref.visible(parents, 8, 1, 2, 2)
    assert np.flatnonzero(see[6]).tolist() == [0, 1, 1 + 5, 1 + 6]
    assert np.flatnonzero(see[0]).tolist() == [0, 1]
    assert tree_ref.words_of(tree_ref.own_visible(parents, 0, 0, 0), 40)[6].tolist() == [0b1100011, 0]
    chain = [tree_ref.CHAIN, 5, 5]
    assert tree_ref.depths(chain) == [0, 1, 2]
    assert tree_ref.visible(None, 3, 2, 2, 1).astype(int).tolist() == [
        [1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    line = [-1, 0, 1, 2, 3]
    for w, s in ((0, 0), (2, 0), (2, 3), (9, 0)):
        assert np.array_equal(tree_ref.visible(line, 5, 1, w, s), tree_ref.visible(None, 5, 1, w, s))
    assert tree_ref.accept(parents, [7, 1, 1, 1, 2, 3, 4, 5], [1, 3, 9, 9, 9, 4, 8, 9]) == ([0, 1, 5, 6], 8)
    assert tree_ref.accept(parents, [7, 1, 1, 1, 2, 3, 4, 5], [6, 3, 9, 9, 9, 4, 8, 9]) == ([0], 6)
    assert tree_ref.accept(chain, [1, 2, 3], [4, 5, 6]) == ([0, 1, 2], 6)
    assert tree_ref.accept([], [], []) == ([], -1)


def test_layers_are_a_list():
    """A cache's layers join, slice and change like any list, and moe_kv_tree_keep takes them as they are then."""
    pytest.importorskip("torch")
    a, b = (m.DeviceKv(2, 4, 6, 16, 1, 64, device="cpu", layers=3) for _ in range(2))
    assert isinstance(a.layers, list) and a.c is a.layers[0]
    a.c.max_blocks = 3
    assert a.layers[0].max_blocks == a.layers.array[0].max_blocks == 3
    both = a.layers + b.layers
    assert [x.pool for x in both] == [p.data_ptr() for p in a.pools + b.pools]
    for x in both:
        x.pool = PTR  # (128-byte aligned)

    def keep(layers):
        return _keep(layers, rows=1, T=0)  # launches nothing

    for layers in (a.layers, both, a.layers[1:], tuple(a.layers), a.layers.array):
        assert keep(layers) == m.MOE_OK
    b.layers[1].kv_heads = 2  # in place
    _refused(m.MOE_EINVAL, lambda: keep(b.layers), "layer 1")
    a.layers[2] = _kv(head_dim=128)  # another struct
    _refused(m.MOE_EINVAL, lambda: keep(a.layers), "layer 2")
    a.layers.pop()
    assert keep(a.layers) == m.MOE_OK
    a.layers.append(_kv(head_dim=128))
    a.layers.append(a.layers[0])
    _refused(m.MOE_EINVAL, lambda: keep(a.layers), "layer 2")
