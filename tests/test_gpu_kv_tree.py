"""GPU tests of drafted trees and sliding windows over the 4-bit key/value cache: what a tree's tokens
see, attention through a view, the kept path, and steps of all of them, against plain 64-bit
restatements (kv_reference.py, kv_tree_reference.py)."""
import numpy as np
import pytest

import kv_reference as ref
import kv_tree_reference as tree_ref
import moe_expert_offload_gb300 as m

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda"


def _np(t):
    return t.detach().cpu().numpy()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _batch(lens, news, T, slots=True):
    """A step's batch as a plan leaves it, slot t for token t."""
    B = len(lens)
    batch = m.DeviceKvBatch(T, B)
    batch.q_start.copy_(_ints(np.concatenate([[0], np.cumsum(news)])))
    batch.kv_len.copy_(_ints(lens))
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, news)] + [np.zeros(0, int)])
    batch.pos[:len(pos)] = _ints(pos)
    return batch


def _parents(rng, news, kinds, max_new):
    rows = []
    for b, n in enumerate(news):
        rows.append(tree_ref.random_parents(rng, n, "chain" if n > max_new else kinds[b % len(kinds)]))
    return rows


def _flat(rows, T, fill):
    flat = [x for r in rows for x in r]
    return _ints(flat + [fill] * (T - len(flat)))


# ------------------------------------------------------------------ plans of trees
ALL_KINDS = ["any", "bushy", "line", "star", "forest", "chain"]


@pytest.mark.parametrize("max_new,news", [
    (1, [1, 1, 0, 1]), (5, [5, 1, 4, 0, 2, 3, 5]), (32, [32, 31, 1, 32, 17, 32, 40]),
    (33, [33, 32, 31, 33, 2, 33]), (64, [64, 63, 33, 64, 64, 64, 300, 0]), (65, [65] * 6),
    (100, [100, 99, 100, 65, 97, 96]), (256, [256, 255, 256, 129, 256, 256, 1000, 1, 0]),
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 9), (1, 0), (1, 4), (2, 0), (7, 3), (31, 60),
                                          (32, 0), (100, 40), (255, 10), (256, 0), (2 ** 31 - 1, 0),
                                          (5, 2 ** 31 - 1)])
def test_tree_plans(max_new, news, window, sinks):
    rng = np.random.default_rng(max_new + window % 1000)
    lens = [n + int(rng.choice([0, 1, 30, 5000])) for n in news]
    T = sum(news) + 3
    rows = _parents(rng, news, ALL_KINDS, max_new)
    batch = _batch(lens, news, T)
    tree = m.DeviceKvTree(T, len(news), max_new)
    tree.parent.copy_(_flat(rows, T, 12345))
    tree.seen.fill_(-7)
    batch.pos[T - 3:] = 99
    before = _np(batch.pos).copy()
    m.moe_kv_tree_plan(batch.c, m.make_view(window, sinks, tree), len(news), T)
    assert int(batch.err[0]) == 0
    seen, pos, start = _np(tree.seen).view(np.uint32), _np(batch.pos), 0
    for L, n, parents in zip(lens, news, rows):
        if n > max_new:
            assert np.all(_np(tree.seen)[start:start + n] == -7)
            assert np.array_equal(pos[start:start + n], before[start:start + n])
        elif n:
            depth = tree_ref.depths(parents)
            see = tree_ref.own_visible(parents, L - n, window, sinks)
            assert np.array_equal(seen[start:start + n, 0], depth)
            assert np.array_equal(seen[start:start + n, 1:], tree_ref.words_of(see, max_new))
            assert np.array_equal(pos[start:start + n], L - n + np.array(depth))
        start += n
    assert np.all(_np(tree.seen)[T - 3:] == -7) and np.all(pos[T - 3:] == 99)


def test_tree_plan_flags_what_does_not_fit():
    """Parents that do not come first, long rows that are no chains, bounds that do not fit."""
    def run(news, lens, rows, max_new=8, T=None, q_start=None):
        T = T or sum(news)
        batch = _batch(lens, news, T)
        if q_start is not None:
            batch.q_start.copy_(_ints(q_start))
        tree = m.DeviceKvTree(T, len(news), max_new)
        tree.parent.copy_(_flat(rows, T, 0))
        tree.seen.fill_(-7)
        m.moe_kv_tree_plan(batch.c, m.make_view(tree=tree), len(news), T)
        return int(batch.err[0]), _np(tree.seen), _np(batch.pos)

    good = [-1, 0, 0, 1]
    for bad in ([-1, 0, 2, 1], [-1, 0, 3, 1], [-1, -3, 0, 1], [0, 0, 0, 1], [-1, 2 ** 31 - 1, 0, 1],
                [-1, -2, 0, 0]):
        err, seen, pos = run([4, 4], [10, 9], [good, bad])
        assert err == m.MOE_DERR_KV_INDEX
        assert seen[:4].tolist() == [[0, 1], [1, 3], [1, 5], [2, 11]]
        mended = [p if -1 <= p < i else -1 for i, p in enumerate(bad)]
        depth = tree_ref.depths(mended)
        words = tree_ref.words_of(tree_ref.own_visible(mended, 5, 0, 0), 8)
        assert seen[4:, 0].tolist() == depth and np.array_equal(seen[4:, 1:], words.view(np.int32))
        assert pos[4:].tolist() == [5 + d for d in depth]
    err, seen, _ = run([9, 4], [9, 4], [[-1] + list(range(8)), good])
    assert err == m.MOE_DERR_KV_INDEX and np.all(seen[:9] == -7) and seen[9, 1] == 1
    for lens, q in (([3, 4], None), ([4, 4], [-1, 4, 8]), ([4, 4], [0, 4, 9]), ([4, -4], None),
                    ([4, 4], [4, 0, 4])):
        err, seen, _ = run([4, 4], lens, [good, good], q_start=q)
        assert err == m.MOE_DERR_KV_INDEX, (lens, q)


# ------------------------------------------------------------------ kept paths
def _choices(rng, rows, hits):
    """Tokens and choices that follow the trees here and there."""
    tokens, nexts = [], []
    for parents in rows:
        n = len(parents)
        tok = rng.integers(0, 5, n)  # few values: siblings with one token
        nxt = rng.integers(5, 9, n)
        if n and parents[0] != tree_ref.CHAIN:
            for c in range(n - 1, 0, -1):
                if 0 <= parents[c] < c and rng.random() < hits:
                    nxt[parents[c]] = tok[c]
        tokens.append(tok.tolist())
        nexts.append(nxt.tolist())
    return tokens, nexts


@pytest.mark.parametrize("max_new,news", [
    (1, [1, 0, 1]), (7, [7, 7, 7, 7, 3, 7, 0]), (33, [33, 33, 33, 33, 33, 33, 100, 2]),
    (256, [256, 256, 256, 200, 256, 256, 5000, 0, 1] * 3),
])
@pytest.mark.parametrize("hits", [0.0, 0.5, 1.0])
def test_accepted_paths(max_new, news, hits):
    rng = np.random.default_rng(max_new)
    rows = _parents(rng, news, ALL_KINDS, max_new)
    tokens, nexts = _choices(rng, rows, hits)
    T, B = sum(news) + 2, len(news)
    batch = _batch([n + 7 for n in news], news, T)
    tree = m.DeviceKvTree(T, B, max_new)
    tree.parent.copy_(_flat(rows, T, -1))
    for t in (tree.path, tree.kept, tree.drop, tree.last):
        t.fill_(77)
    m.moe_kv_tree_accept(batch.c, tree.c, B, T, _flat(tokens, T, 0), _flat(nexts, T, 0), tree.path,
                         tree.kept, tree.drop, tree.last)
    assert int(batch.err[0]) == 0
    path, start = _np(tree.path), 0
    longest = 0
    for b, (n, parents) in enumerate(zip(news, rows)):
        want, last = tree_ref.accept(parents, tokens[b], nexts[b])
        assert path[start:start + n].tolist() == want + [-1] * (n - len(want))
        got = [int(t[b]) for t in (tree.kept, tree.drop, tree.last)]
        assert got == [len(want), len(want) - n, last], b
        if parents and parents[0] != tree_ref.CHAIN:
            longest = max(longest, len(want))
        start += n
    assert path[start:].tolist() == [77, 77]
    if hits == 1.0 and max_new >= 7:
        assert longest == max_new  # the line, taken to its end


def test_accept_flags_what_does_not_fit():
    rows = [[-1, 0, 2, 1], [-1, 0, 0, 1], [-1, 0, 1, 2, 3]]
    news, T = [4, 4, 5], 13
    batch = _batch([4, 4, 5], news, T)
    tree = m.DeviceKvTree(T, 3, 4)
    tree.parent.copy_(_flat(rows, T, 0))
    tok = _ints([1] * T)
    m.moe_kv_tree_accept(batch.c, tree.c, 3, T, tok, tok, tree.path, tree.kept, tree.drop, tree.last)
    assert int(batch.err[0]) == m.MOE_DERR_KV_INDEX
    # token 2 follows itself and is never kept; token 3's parent is a good one
    assert _np(tree.path).tolist() == [0, 1, 3, -1, 0, 1, 3, -1, 0, 1, 2, 3, 4]
    assert _np(tree.kept).tolist() == [3, 3, 5] and _np(tree.drop).tolist() == [-1, -1, 0]
    batch.err.zero_()
    batch.kv_len[1] = 3  # fewer tokens than new ones
    tree.path.fill_(9)
    m.moe_kv_tree_accept(batch.c, tree.c, 2, T, tok, tok, tree.path, tree.kept, tree.drop, tree.last)
    assert int(batch.err[0]) == m.MOE_DERR_KV_INDEX
    assert _np(tree.kept)[:2].tolist() == [3, 0] and _np(tree.drop)[:2].tolist() == [-1, 0]
    assert _np(tree.last)[:2].tolist() == [1, -1] and torch.all(tree.path[4:] == 9)


# ------------------------------------------------------------------ keys and values moved
def _pools(layers, blocks, P, K, D, width, rows, seed):
    kv = m.DeviceKv(rows, width, blocks, P, K, D, layers=layers)
    g = torch.Generator(device=DEV).manual_seed(seed)
    for p in kv.pools:
        p.copy_(torch.randint(0, 256, p.shape, generator=g, device=DEV, dtype=torch.uint8))
    return kv


def _token_bytes(pool, slot, K, P, D):
    """The bytes of one token in a pool: codes, scales and biases of K and V, all heads."""
    flat, G, out = pool.reshape(-1), D // 64, []
    col = np.arange(0, D, 2)
    for h in range(K):
        base = ((slot // P * K + h) * (P // 16) + slot % P // 16) * 18 * D
        key, g = slot % 16, np.arange(G)
        at = [base + ref.code_byte(D, key, col), base + 8 * D + ref.code_byte(D, key, col)]
        for part in (0, 1):
            for i in (part * 16 * G + key * G + g, 32 * G + part * 16 * G + g * 16 + key):
                at += [base + 16 * D + 2 * i, base + 16 * D + 2 * i + 1]
        out.append(np.concatenate(at))
    return np.concatenate(out)


@pytest.mark.parametrize("layers,P,K,D,paths", [
    (1, 64, 2, 256, [(16, [0, 3, 9])]),
    (3, 16, 8, 128, [(64, [0, 1, 2, 7, 30, 63]), (5, [0, 1, 2, 3, 4]), (0, []), (9, [0])]),
    (2, 32, 5, 64, [(40, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 20, 30, 39]), (33, list(range(16, 33))),
                    (256, list(range(0, 256, 2))), (256, list(range(1, 256)))]),
    (2, 128, 3, 256, [(256, [0] + list(range(20, 250, 3))), (2, [1]), (1, [0])]),
    (130, 16, 1, 64, [(20, [0, 2, 19]), (17, [5, 16])]),
    (1, 16, 1, 128, [(3000, list(range(0, 3000, 3)))]),  # a caller's own path of a long row
])
def test_kept_tokens_move(layers, P, K, D, paths):
    rng = np.random.default_rng(layers + D)
    news = [n for n, _ in paths]
    T, B = sum(news) + 2, len(news)
    blocks = -(-T // P) + 3
    kv = _pools(layers, blocks, P, K, D, 4, B, layers)
    batch = _batch([n + 40 for n in news], news, T)
    slots = rng.permutation(blocks * P)[:T]
    batch.slot.copy_(_ints(slots))
    path = np.full(T, -1)
    start = 0
    for n, p in paths:
        path[start:start + len(p)] = p
        start += n
    want = [_np(p).copy() for p in kv.pools]
    for pool in want:
        old, start = pool.copy(), 0
        for n, p in paths:
            for i, a in enumerate(p):
                src = _token_bytes(pool, slots[start + a], K, P, D)
                dst = _token_bytes(pool, slots[start + i], K, P, D)
                pool.reshape(-1)[dst] = old.reshape(-1)[src]
            start += n
    m.moe_kv_tree_keep(kv.layers, batch.c, B, T, _ints(path), _ints([len(p) for _, p in paths]))
    assert int(batch.err[0]) == 0
    for l, (got, w) in enumerate(zip(kv.pools, want)):
        assert np.array_equal(_np(got), w), l


def test_keep_leaves_bad_rows_as_they_are():
    P, K, D, n = 16, 2, 128, 6
    bad = [([0, 2, 2], 3), ([0, 3, 1], 3), ([0, 2, 6], 3), ([-1, 2, 3], 3), ([0, 2, 5], 7),
           ([0, 2, 5], -1), ([0, 2 ** 31 - 1, 5], 3)]
    kv = _pools(2, 12, P, K, D, 4, 2, 1)
    before = [_np(p).copy() for p in kv.pools]
    for p, count in bad:
        batch = _batch([20, 20], [n, n], 2 * n)
        batch.slot.copy_(_ints(np.arange(2 * n) * 7))
        path = [0, 1, 2, 3, 4, 5] + p + [-1] * 3
        m.moe_kv_tree_keep(kv.layers, batch.c, 2, 2 * n, _ints(path), _ints([2, count]))
        assert int(batch.err[0]) == m.MOE_DERR_KV_INDEX, (p, count)
        for got, w in zip(kv.pools, before):
            assert np.array_equal(_np(got), w), (p, count)
    # slots outside the pool: those tokens are not moved, the others are
    for outside in (12 * P, -1, -2 ** 31, 2 ** 31 - 1):
        for at in (1, 2, 4):  # a place; a place and a source; a source
            batch = _batch([20], [n], n)
            slots = np.arange(n) * 7
            slots[at] = outside
            batch.slot.copy_(_ints(slots))
            want = [w.copy() for w in before]
            for w in want:
                old = w.copy()
                for i, a in enumerate([0, 2, 4]):
                    if at not in (i, a):
                        w.reshape(-1)[_token_bytes(w, slots[i], K, P, D)] = old.reshape(-1)[
                            _token_bytes(w, slots[a], K, P, D)]
            for p, b in zip(kv.pools, before):
                p.copy_(torch.tensor(b, device=DEV))
            m.moe_kv_tree_keep(kv.layers, batch.c, 1, n, _ints([0, 2, 4, -1, -1, -1]), _ints([3]))
            assert int(batch.err[0]) == m.MOE_DERR_KV_INDEX
            for got, w in zip(kv.pools, want):
                assert np.array_equal(_np(got), w), (outside, at)


# ------------------------------------------------------------------ attention
def _fill(kv, D, gen):
    """Random codes, scales and biases in every tile of the pool."""
    tiles = kv.pool.view(-1, 18 * D)
    n, G = tiles.shape[0], D // 64
    tiles[:, : 16 * D] = torch.randint(0, 256, (n, 16 * D), generator=gen, device=DEV,
                                       dtype=torch.uint8)
    s = 0.1 + 0.3 * torch.rand(2, n, 16 * G, generator=gen, device=DEV)
    b = -7.5 * s + 0.3 * torch.randn(2, n, 16 * G, generator=gen, device=DEV)
    tiles[:, 16 * D:] = torch.cat((s[0], b[0], s[1], b[1]), 1).half().view(torch.uint8)


def _poison(kv, K, P, D, live):
    """NaN in the scales and biases of every slot that is not live."""
    G, blocks = D // 64, kv.pool.shape[0]
    mask = np.ones(blocks * P, bool)
    mask[live] = False
    meta = kv.pool.view(-1, 18 * D)[:, 16 * D:].contiguous().view(torch.float16)
    dead = torch.tensor(mask, device=DEV).view(blocks, 1, P // 16, 16).expand(-1, K, -1, -1)
    dead = dead.reshape(-1, 16)
    parts = meta.view(-1, 4, 16 * G)
    by_key = dead[:, :, None].expand(-1, 16, G).reshape(-1, 16 * G)
    by_group = dead[:, None, :].expand(-1, G, 16).reshape(-1, 16 * G)
    for i in range(4):
        parts[:, i].masked_fill_(by_key if i < 2 else by_group, float("nan"))
    kv.pool.view(-1, 18 * D)[:, 16 * D:] = meta.view(torch.uint8)


def _case(P, K, D, r, lens, news, window, sinks, kinds=None, max_tree=None, seed=0, poison=False,
          heavy=0, idle=0):
    """A cache of random tokens and a step's queries; kinds None: no tree, every row a chain.
    heavy: so many longer rows follow (which kernel takes which rows goes by the batch's work), with
    as many new tokens as one tile of queries holds where the others have no more; idle: so many
    rows without new tokens.  poison: every slot that no new token sees is NaN, and the blocks of which none is seen have
    ids outside the pool."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    many = 128 // r if max(news) * r <= 128 else 200
    lens, news = lens + [1500] * heavy + [0] * idle, news + [many] * heavy + [0] * idle
    B, width = len(lens), max(1, -(-max(lens) // P)) + 1
    blocks = sum(-(-n // P) for n in lens) + 3
    kv = m.DeviceKv(B, width, blocks, P, K, D)
    T = sum(news) + 2
    batch = _batch(lens, news, T)
    order = rng.permutation(blocks)
    table = np.full((B, width), -1)
    used = 0
    for b, n in enumerate(lens):
        k = -(-n // P)
        table[b, :k] = order[used:used + k]
        used += k
    _fill(kv, D, gen)
    tree, rows = None, [None] * B
    if kinds:
        max_tree = max_tree or max(1, max(news))
        tree = m.DeviceKvTree(T, B, max_tree)
        rows = _parents(rng, news, kinds, max_tree)
        tree.parent.copy_(_flat(rows, T, -1))
    see = [tree_ref.visible(rows[b], n, L - n, window, sinks) if n else np.zeros((0, L), bool)
           for b, (L, n) in enumerate(zip(lens, news))]
    shown = table.copy()
    if poison:
        live = []
        for b, s in enumerate(see):
            j = np.flatnonzero(s.any(0))
            live.append(table[b, j // P] * P + j % P)
            unseen = np.setdiff1d(np.arange(width), j // P)
            shown[b, unseen] = rng.choice([-1, blocks, 2 ** 31 - 1, -2 ** 31], len(unseen))
        _poison(kv, K, P, D, np.concatenate(live))
    kv.block_table.copy_(_ints(shown))
    q = (torch.randn(T, K * r, D, generator=gen, device=DEV) * 1.5).bfloat16()
    c = dict(kv=kv, batch=batch, q=q, T=T, H=K * r, K=K, D=D, P=P, B=B, lens=lens, news=news,
             table=table, scale=D ** -0.5, max_new=max(1, max(news)), see=see, tree=tree,
             view=m.make_view(window, sinks, tree))
    if tree:
        m.moe_kv_tree_plan(batch.c, c["view"], B, T)
    return c


def _run(c, q=None, ws=None, stream=None, out=None, max_new=None):
    max_new = max_new or c["max_new"]
    if out is None:
        out = torch.full_like(c["q"], 5.0)
    n = m.moe_kv_attention_workspace_bytes(c["kv"].c, c["B"], c["T"], c["H"], max_new)
    if ws is None:
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # NaN in every float
    m.moe_kv_attention_view(c["kv"].c, c["batch"].c, c["view"], c["B"], c["q"] if q is None else q,
                            c["T"], c["H"], max_new, c["scale"], ws, n, out, stream)
    return out


def _check(c, out, rows=None):
    pool, got, q = _np(c["kv"].pool), _f64(out), _f64(c["q"])
    start, want_all, got_all = 0, [], []
    for b, (L, n) in enumerate(zip(c["lens"], c["news"])):
        if n and (rows is None or b in rows):
            j = np.flatnonzero(c["see"][b].any(0))
            k, v = ref.read_slots(pool, c["table"][b, j // c["P"]] * c["P"] + j % c["P"], c["K"],
                                  c["P"], c["D"])
            qq = q[start:start + n]
            want = tree_ref.attention(qq, k, v, c["scale"], c["see"][b][:, j])
            tol = ref.attention_bound(qq, k, v, c["scale"], want)
            g = got[start:start + n]
            assert np.all(np.isfinite(g)), f"row {b}: not finite"
            off = np.abs(g - want)
            assert np.all(off <= tol), (b, L, n, float((off - tol).max()), float(off.max()))
            want_all.append(want.ravel())
            got_all.append(g.ravel())
        start += n
    if want_all:
        w, g = np.concatenate(want_all), np.concatenate(got_all)
        rel = np.linalg.norm(g - w) / np.linalg.norm(w)
        assert rel <= ref.ATTENTION_REL, rel
    assert torch.all(out[sum(c["news"]):] == 5.0), "rows behind the last token changed"


WINDOWS = [
    # P, kv heads, D, group, lengths, new tokens, window, sinks
    (64, 2, 256, 8, [1000], [1], 128, 4),
    (16, 1, 64, 1, [1], [1], 1, 0),
    (16, 2, 128, 8, [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 300], [1] * 11, 16, 0),
    (16, 2, 128, 8, [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 300], [1] * 11, 17, 1),
    (16, 2, 64, 8, [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 300], [1] * 11, 1, 16),
    (32, 1, 256, 4, [127, 128, 129, 5, 700], [1] * 5, 33, 40),
    (32, 8, 64, 4, [3, 0, 257, 0, 40, 900], [1, 0, 1, 0, 1, 1], 64, 3),
    (64, 4, 128, 6, [513, 100, 2000], [1, 1, 1], 500, 70),
    (32, 4, 128, 8, [400, 4, 129, 64, 9, 1000], [4, 4, 2, 1, 3, 8], 3, 2),
    (64, 2, 256, 8, [100, 2000], [3, 4], 100, 0),
    (64, 2, 256, 8, [257], [257], 20, 0),
    (16, 2, 128, 8, [130, 1500], [130, 700], 100, 4),
    (64, 2, 128, 8, [640, 128], [128, 100], 1, 0),
    (64, 2, 128, 8, [640, 128], [128, 100], 129, 17),
    (128, 2, 64, 1, [300, 17, 1290], [300, 17, 1000], 128, 4),
    (16, 1, 256, 6, [333, 1000], [200, 700], 48, 130),
    (64, 1, 128, 5, [1500, 64], [70, 64], 1000, 0),
    (64, 2, 256, 16, [200, 900, 0, 50], [200, 1, 0, 33], 60, 33),
    (32, 2, 128, 4, [3000, 40, 2100, 1], [5, 40, 300, 1], 257, 16),
    (64, 8, 64, 2, [1256], [1256], 300, 0),
    (64, 8, 64, 2, [256], [256], 2 ** 31 - 1, 2 ** 31 - 1),
    (16, 1, 128, 64, [700, 9], [1, 2], 100, 1),
    (16, 1, 256, 64, [700, 90], [1, 2], 100, 600),
]


# heavy rows, idle rows, poison: little work (the decode kernel takes it), and enough for the prompt
# kernel, which finds its shares in another way from 32 rows on
ROWS = [(0, 0, False), (0, 0, True), (14, 0, True), (14, 40, False)]


@pytest.mark.parametrize("i", range(len(WINDOWS)))
@pytest.mark.parametrize("heavy,idle,poison", ROWS)
def test_windows(i, heavy, idle, poison):
    P, K, D, r, lens, news, window, sinks = WINDOWS[i]
    c = _case(P, K, D, r, lens, news, window, sinks, seed=200 + i, poison=poison, heavy=heavy,
              idle=idle)
    out = _run(c)
    assert int(c["batch"].err[0]) == 0
    _check(c, out, rows=range(len(lens) + min(heavy, 1)))


TREES = [
    # P, kv heads, D, group, lengths, new tokens, window, sinks, kinds, the longest tree
    (64, 2, 256, 8, [1000], [4], 0, 0, ["any"], 4),
    (16, 2, 128, 8, [8, 15, 16, 17, 31, 32, 33, 63, 64, 65], [8, 1, 7, 8, 8, 2, 8, 8, 3, 8], 0, 0, ALL_KINDS, 8),
    (16, 4, 64, 1, [64, 100, 333, 65], [64, 63, 33, 64], 0, 0, ["any", "bushy", "forest"], 64),
    (32, 1, 128, 2, [32, 1000, 47, 48], [32, 31, 32, 32], 0, 0, ["forest", "line", "star", "any"], 256),
    (64, 2, 256, 8, [300, 20], [20, 16], 0, 0, ["any"], 20),
    (64, 2, 128, 8, [64, 900, 129], [64, 60, 64], 0, 0, ["any", "star", "forest"], 64),
    (16, 1, 128, 4, [256, 700, 300], [256, 255, 129], 0, 0, ["any", "forest", "bushy"], 256),
    (128, 2, 64, 4, [500, 256], [200, 256], 0, 0, ["bushy", "any"], 256),
    (32, 1, 256, 16, [400, 30, 100], [40, 30, 1], 0, 0, ["bushy", "line", "chain"], 100),
    # windows shorter and longer than the trees' depth, sinks before, across and behind the cached tokens
    (16, 2, 128, 8, [8, 300, 17, 900], [8, 8, 8, 8], 3, 0, ["line", "any"], 8),
    (16, 2, 64, 2, [30, 300, 32, 900], [30, 30, 32, 7], 5, 4, ["line", "bushy", "forest"], 32),
    (64, 2, 256, 4, [8, 300, 9], [8, 8, 8], 2, 5, ["line", "bushy"], 8),
    (16, 1, 128, 8, [100, 1000, 70], [100, 90, 64], 20, 90, ["line", "bushy", "forest"], 100),
    (64, 2, 256, 16, [300, 1000, 33], [33, 30, 33], 100, 4, ["any", "line"], 40),
    (32, 4, 64, 8, [700, 64], [64, 64], 1, 0, ["any", "line"], 64),
    (16, 1, 256, 3, [280, 1200], [256, 200], 48, 20, ["bushy", "line"], 256),
    # chains, prompts and trees in one call
    (32, 2, 128, 4, [3000, 40, 2100, 1, 500, 600], [5, 40, 300, 1, 64, 90], 0, 0, ["any", "chain"], 64),
    (32, 2, 128, 4, [3000, 40, 2100, 1, 500, 600], [5, 40, 300, 1, 64, 90], 150, 4, ["any", "chain"], 64),
    (16, 1, 64, 8, [900, 33, 64], [400, 33, 7], 100, 0, ["forest"], 32),
]


@pytest.mark.parametrize("i", range(len(TREES)))
@pytest.mark.parametrize("heavy,idle,poison", ROWS)
def test_trees(i, heavy, idle, poison):
    P, K, D, r, lens, news, window, sinks, kinds, longest = TREES[i]
    c = _case(P, K, D, r, lens, news, window, sinks, kinds, longest, seed=300 + i, poison=poison,
              heavy=heavy, idle=idle)
    out = _run(c)
    assert int(c["batch"].err[0]) == 0
    _check(c, out, rows=range(len(lens) + min(heavy, 1)))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 2000])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("r,news", [(4, [32, 31, 17, 32]), (4, [60, 40, 256, 200]), (8, [130, 1, 100, 256])])
@pytest.mark.parametrize("heavy,idle", [(0, 0), (14, 0), (14, 40)])
def test_trees_under_windows_past_every_position(window, D, r, news, heavy, idle):
    """Windows up to the largest there is leave everything in a tree's sight: bushy trees and stars, whose late
    tokens stand far behind their position."""
    lens = [n + x for n, x in zip(news, (0, 700, 30, 333))]
    c = _case(16, 2, D, r, lens, news, window, 0, ["star", "bushy", "star", "forest"], 256, seed=61,
              heavy=heavy, idle=idle)
    out = _run(c)
    assert int(c["batch"].err[0]) == 0
    _check(c, out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news", [[1, 2, 1], [90, 3, 70]])
@pytest.mark.parametrize("heavy", [0, 14])
def test_a_view_of_everything_is_plain_attention(D, news, heavy):
    """Without a window and a tree the results are moe_kv_attention's, bit for bit; windows past every
    row, or sinks, leave everything visible too."""
    c = _case(32, 2, D, 4, [900, 60, 333], news, 0, 0, seed=D, heavy=heavy)
    out = torch.full_like(c["q"], 5.0)
    n = m.moe_kv_attention_workspace_bytes(c["kv"].c, c["B"], c["T"], c["H"], c["max_new"])
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    m.moe_kv_attention(c["kv"].c, c["batch"].c, c["B"], c["q"], c["T"], c["H"], c["max_new"],
                       c["scale"], ws, n, out)
    assert torch.equal(_run(c), out)
    for window, sinks in ((1500, 0), (2 ** 31 - 1, 7), (0, 50), (1, 1500)):
        c["view"] = m.make_view(window, sinks)
        got = _run(c)
        _check(c, got, rows=range(3))
        if window == 0:
            assert torch.equal(got, out)


def _wide_case(P, K, D, r, lens, news, window, sinks, cycle, seed, kinds=None):
    """Rows that all read one context, whose blocks come again after `cycle` of them, so that long
    contexts need a small pool."""
    c = _case(P, K, D, r, [cycle * P] + [1] * (len(lens) - 1), [1] * len(lens), 0, 0, seed=seed)
    order = c["table"][0, :cycle]
    width = -(-max(lens) // P)
    c["table"] = np.tile(order[np.arange(width) % cycle], (len(lens), 1))
    kv = c["kv"]
    kv.block_table = _ints(c["table"])
    kv.c.block_table, kv.c.max_blocks = kv.block_table.data_ptr(), width
    rng = np.random.default_rng(seed)
    c["T"] = T = sum(news) + 2
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c["q"] = (torch.randn(T, K * r, D, generator=gen, device=DEV) * 1.5).bfloat16()
    c["batch"], c["lens"], c["news"], c["max_new"] = _batch(lens, news, T), lens, news, max(news)
    c["rows"], tree = [None] * len(lens), None
    if kinds:
        tree = c["tree"] = m.DeviceKvTree(T, len(lens), max(news))
        c["rows"] = _parents(rng, news, kinds, max(news))
        tree.parent.copy_(_flat(c["rows"], T, -1))
    c["view"] = m.make_view(window, sinks, tree)
    if tree:
        m.moe_kv_tree_plan(c["batch"].c, c["view"], len(lens), T)
    return c


def _check_wide(c, out, window, sinks):
    """_check in 64 bits on the GPU, of a context that all rows share."""
    P, K, D, r = c["P"], c["K"], c["D"], c["H"] // c["K"]
    slots = np.arange(c["kv"].pool.shape[0] * P)
    k_all, v_all = (torch.tensor(x, device=DEV) for x in
                    ref.read_slots(_np(c["kv"].pool), slots, K, P, D))
    big = v_all.abs().amax(0).view(K, -1, 64).amax(-1).repeat_interleave(64, 1)  # [K, D]
    start, wrong, size = 0, 0.0, 0.0
    for b, (L, n) in enumerate(zip(c["lens"], c["news"])):
        base = L - n
        low = max(0, base - window + 1) if window else 0
        j = np.concatenate((np.arange(min(sinks, low)), np.arange(low, L)))
        parents = c["rows"][b] or [tree_ref.CHAIN] + [0] * (n - 1)
        depth = np.array(tree_ref.depths(parents))[:, None]
        old = j[j < base][None]
        see = np.ones((n, old.shape[1]), bool)
        if window:
            see = (old > base + depth - window) | (old < sinks)
        see = torch.tensor(np.concatenate((see, tree_ref.own_visible(parents, base, window, sinks)), 1), device=DEV)
        at = torch.tensor(c["table"][0][j // P] * P + j % P, device=DEV)
        for h in range(K):
            k, v = k_all[at, h], v_all[at, h]
            q = c["q"][start:start + n, h * r:(h + 1) * r].double()  # [n, r, D]
            x = (q @ k.T * c["scale"]).masked_fill(~see[:, None], -np.inf)
            want = torch.softmax(x, -1) @ v
            spread = c["scale"] * (q.square() @ k.square().T).amax(-1, True).sqrt() * 2.0 ** -11
            tol = (want.abs() * 2.0 ** -8 + 1e-6
                   + 2 * big[h] * (4 * 2.0 ** -11 + 2 * 8 * spread / 3 ** 0.5))
            got = out[start:start + n, h * r:(h + 1) * r].double()
            off = (got - want).abs()
            assert bool((off <= tol).all()), (L, n, h, float((off / tol).max()))
            wrong, size = wrong + float(off.square().sum()), size + float(want.square().sum())
        start += n
    assert (wrong / size) ** 0.5 <= ref.ATTENTION_REL
    assert torch.all(out[start:] == 5.0)


@pytest.mark.parametrize("P,K,D,r,B,least,most,n,window,sinks,cycle,kinds", [
    # decode rows: windows of a few tiles over many rows, and long ones over few
    (64, 8, 128, 4, 200, 150, 8191, 1, 1024, 4, 128, None),
    (16, 2, 256, 8, 8, 129000, 131071, 1, 32768, 64, 300, None),
    (32, 4, 64, 3, 100, 4000, 9000, 3, 2500, 300, 282, None),
    (128, 2, 128, 16, 12, 20000, 30001, 2, 9999, 0, 40, None),
    # prompts
    (64, 2, 256, 8, 2, 9000, 9400, 2600, 700, 4, 148, None),
    (64, 4, 128, 8, 1, 13001, 13001, 3000, 4096, 0, 210, None),
    (16, 8, 64, 1, 5, 8000, 9000, 4000, 129, 1000, 563, None),
    # trees
    (64, 8, 128, 4, 40, 150, 8191, 16, 0, 0, 128, ["any", "bushy"]),
    (64, 4, 128, 4, 20, 3000, 8191, 64, 1500, 4, 128, ["any", "line"]),
    (16, 2, 256, 8, 6, 9000, 20000, 50, 0, 0, 300, ["bushy"]),
    (32, 8, 64, 2, 30, 900, 9000, 200, 0, 0, 282, ["any", "forest"]),
])
def test_views_of_long_contexts(P, K, D, r, B, least, most, n, window, sinks, cycle, kinds):
    """Work enough that every warp (CTA) turns its buffers many times over and units are cut, the
    gap between sinks and window among what it passes."""
    rng = np.random.default_rng(P + D)
    lens = rng.integers(least, most + 1, B).tolist()
    news = [min(L, n) for L in lens]
    c = _wide_case(P, K, D, r, lens, news, window, sinks, cycle, 35, kinds)
    out = _run(c)
    assert int(c["batch"].err[0]) == 0
    _check_wide(c, out, window, sinks)
    assert torch.equal(_run(c), out)


def _longest(c, cycle):
    """The case's one row on a table as wide as there can be, over `cycle` blocks of 16 tokens."""
    kv, width = c["kv"], (2 ** 31 - 1) // 16
    c["table"] = np.resize(c["table"][0, :cycle].astype(np.int32), (1, width))
    kv.block_table = torch.tensor(c["table"], device=DEV)
    kv.c.block_table, kv.c.max_blocks = kv.block_table.data_ptr(), width


@pytest.mark.parametrize("D,r,n,window,sinks,kinds", [
    (64, 16, 1000, 1000, 20, None), (128, 16, 1000, 1000, 20, None), (256, 16, 1000, 1000, 0, None),
    (128, 32, 256, 500, 4, ["bushy"]), (64, 32, 256, 500, 4, ["star"]), (256, 32, 256, 500, 0, ["forest"]),
    (128, 8, 1, 1000, 20, None), (256, 4, 5, 300, 0, ["any"]),
])
def test_views_up_to_the_last_position(D, r, n, window, sinks, kinds):
    """Rows that end at the last positions that there can be: what lies behind them passes 2^31 - 1."""
    cycle = 40
    c = _wide_case(16, 1, D, r, [n + 900], [n], window, sinks, cycle, 7, kinds)
    _longest(c, cycle)
    for less in (0, 1, 16, 47, 84, 112, 128, 300):
        L = 2 ** 31 - 16 - less
        c["lens"], c["batch"] = [L], _batch([L], [n], c["T"])
        if kinds:
            m.moe_kv_tree_plan(c["batch"].c, c["view"], 1, c["T"])
        out = _run(c)
        assert int(c["batch"].err[0]) == 0
        _check_wide(c, out, window, sinks)


def test_a_whole_context_of_the_last_position():
    """A causal row that sees 2^31 - 16 keys, whose values are all 1.5: so are its results, but for the sums'
    roundings.  A CTA adds up 2^24 / 152 = 110400 blocks of 128 keys: the weights' sum to the nearest (2^-24
    each, 0.7%), the products in eight steps that may lose a whole one of 2^-23 (10.5%), and bf16's 2^-8."""
    D, n, cycle = 64, 8, 40
    c = _wide_case(16, 1, D, 16, [n + 900], [n], 0, 0, cycle, 7)
    meta = c["kv"].pool.view(-1, 18 * D)[:, 16 * D:].view(torch.float16)  # scales and biases of K, of V
    meta[:, 32:48], meta[:, 48:] = 0.0, 1.5
    _longest(c, cycle)
    L = 2 ** 31 - 16
    c["lens"], c["batch"] = [L], _batch([L], [n], c["T"])
    out = _run(c)
    assert int(c["batch"].err[0]) == 0
    assert float((out[:n].float() / 1.5 - 1).abs().max()) <= 0.12
    assert torch.all(out[n:] == 5.0)


@pytest.mark.parametrize("B", [31, 32, 33, 600, 1000])
@pytest.mark.parametrize("D,window", [(64, 20), (256, 0), (128, 50)])
def test_views_of_row_counts(B, D, window):
    """Around the row counts where the shares are found in another way: trees, idle rows and prompts."""
    rng = np.random.default_rng(B + D)
    lens = rng.integers(0, 90, B)
    news = np.minimum(lens, rng.integers(0, 9, B))
    lens[B // 2], news[B // 2] = 400, 130
    lens[B - 1], news[B - 1] = 140, 140
    c = _case(16, 1, D, 4, lens.tolist(), news.tolist(), window, 3 if window else 0, ALL_KINDS, 16,
              seed=70 + B, poison=True)
    out = _run(c)
    assert int(c["batch"].err[0]) == 0
    _check(c, out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kinds,idle", [(None, 0), (["any", "chain", "bushy"], 100)])
def test_views_of_many_units_of_one_block(D, kinds, idle):
    """Hundreds of rows of up to 128 queries per kv head in a short window: their units are one block of
    keys each, several on a CTA, of which (head_dim 64 and 128) the second query tile has none."""
    rng = np.random.default_rng(D)
    news = rng.integers(28, 33, 400).tolist()
    lens = [n + int(x) for n, x in zip(news, rng.integers(0, 500, 400))]
    c = _case(16, 2, D, 4, lens, news, 60, 4, kinds, 32, seed=90 + D, idle=idle)
    out = _run(c)
    assert int(c["batch"].err[0]) == 0
    _check(c, out)
    for _ in range(20):
        again = _run(c)
        assert int(c["batch"].err[0]) == 0 and torch.equal(again, out)


@pytest.mark.parametrize("size", [1e2, 1e4, 1e9, 1e30])
@pytest.mark.parametrize("D,news", [(D, n) for D in (64, 128, 256) for n in ([130, 60, 33], [1, 4, 2])])
@pytest.mark.parametrize("heavy", [0, 14])
def test_views_of_far_scores(D, news, size, heavy):
    """Scores far from zero on both sides: results stay finite and within the visible values' hull."""
    c = _case(32, 1, D, 8, [500, 260, 33], news, 40, 2, ["any", "line"], 64, seed=31, heavy=heavy)
    q = (c["q"].float() * size).bfloat16()
    out = _run(c, q=q)
    assert int(c["batch"].err[0]) == 0
    got, pool, start = _f64(out), _np(c["kv"].pool), 0
    for b, (L, n) in enumerate(zip(c["lens"][:4], c["news"])):
        for i in range(n):
            j = np.flatnonzero(c["see"][b][i])
            _, v = ref.read_slots(pool, c["table"][b, j // 32] * 32 + j % 32, 1, 32, D)
            slack = np.abs(v).max() * 2.0 ** -7
            g = got[start + i]
            assert np.all(np.isfinite(g))
            assert np.all(g >= v.min(0) - slack) and np.all(g <= v.max(0) + slack), (b, i)
        start += n


@pytest.mark.parametrize("news", [[1, 8], [120, 100]])
@pytest.mark.parametrize("heavy", [0, 14])
@pytest.mark.parametrize("D", [128, 256])
def test_views_leave_out_bad_blocks_and_rows(news, heavy, D):
    c = _case(16, 2, D, 4, [300, 270], news, 200, 20, ["any"], 256, seed=17, heavy=heavy)
    good = _run(c)
    assert int(c["batch"].err[0]) == 0
    c["kv"].block_table[1, 10] = c["kv"].pool.shape[0]  # seen by row 1
    out = _run(c)
    assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
    assert torch.equal(out[:news[0]], good[:news[0]]) and torch.all(torch.isfinite(out.float()))
    assert not torch.equal(out[news[0]:sum(news)], good[news[0]:sum(news)])
    c["kv"].block_table[1].fill_(-1)  # not a key is left
    out = _run(c)
    assert not torch.any(out[news[0]:sum(news)]) and torch.equal(out[:news[0]], good[:news[0]])
    for value in (c["kv"].c.max_blocks * 16 + 1, -1, news[1] - 1):
        c["batch"].err.zero_()
        c["batch"].kv_len[1] = value
        out = _run(c)
        assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
        assert torch.all(out[news[0]:sum(news)] == 5.0)
        _check(c, out, rows=[0])  # (its work may be shared out in another way without row 1's)


@pytest.mark.parametrize("heavy", [0, 14])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("window,sinks,kinds", [(37, 2, None), (200, 20, ["any"]), (150, 0, ["line"])])
def test_views_without_a_block(heavy, D, P, window, sinks, kinds):
    """Blocks outside the pool where a row's window begins (within a tile), in its middle, at its end
    and under its sinks: their keys alone are left out."""
    lens, news = [900, 523, 333], [5, 90, 30]
    c = _case(P, 2, D, 4, lens, news, window, sinks, kinds, 256, seed=47, heavy=heavy)
    for b, (L, n) in enumerate(zip(lens, news)):
        base = L - n
        spots = [[max(0, base - window + 1) // P], [(base - 1) // P], [(L - 1) // P, 0]][b]
        for i in spots:
            c["kv"].block_table[b, i] = [-1, c["kv"].pool.shape[0], 2 ** 31 - 1][b]
            c["see"][b][:, i * P:(i + 1) * P] = False
    out = _run(c)
    assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
    start, pool = 0, _np(c["kv"].pool)
    for b, (L, n) in enumerate(zip(lens, news)):
        j = np.arange(L)
        k, v = ref.read_slots(pool, c["table"][b, j // P] * P + j % P, 2, P, D)
        q, got, see = _f64(c["q"])[start:start + n], _f64(out)[start:start + n], c["see"][b]
        left = see.any(1)  # a token that is left without a key is 0
        assert not got[~left].any()
        want = tree_ref.attention(q[left], k, v, c["scale"], see[left])
        tol = ref.attention_bound(q[left], k, v, c["scale"], want)
        assert np.all(np.abs(got[left] - want) <= tol), b
        start += n


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heavy", [0, 14])
@pytest.mark.parametrize("D,news", [(64, [20, 9, 30]), (128, [20, 9, 30]), (128, [90, 1, 70]), (256, [20, 9, 30])])
def test_broken_values_and_queries_stay_where_they_are(D, news, heavy, bad):
    """A value's scale that is NaN or infinite spoils the row that sees it and no other, one outside the
    window no row; a broken query spoils its own result and no other."""
    c = _case(16, 2, D, 4, [250, 300, 120], news, 60, 2, ["any"], 200, seed=53, heavy=heavy)
    good = _run(c)
    meta = c["kv"].pool.view(-1, 18 * D)[:, 16 * D:].view(torch.float16)  # [tile][part][...]
    G, base = D // 64, 250 - news[0]
    for at, seen in ((base - 62, False), (base - 5, True)):
        tile = int(c["table"][0, at // 16]) * 2 + 1  # row 0, kv head 1
        meta[tile, 2 * 16 * G + at % 16] = bad  # V scale of group 0
        out = _run(c)
        assert int(c["batch"].err[0]) == 0
        _check(c, out, rows=[1, 2])
        row = out[:news[0]].float()
        assert torch.isfinite(row[:, :4]).all()
        assert torch.isfinite(row[:, 4:, :64]).all() != seen
        if not seen:
            assert torch.equal(out, good)
    c = _case(16, 2, D, 4, [250, 300, 120], news, 60, 2, ["any"], 200, seed=53, heavy=heavy)
    q = c["q"].clone()
    q[3, 1, 7], q[sum(news) - 1, 5, 0] = bad, bad
    out = _run(c, q=q)
    touched = torch.zeros(c["T"], c["H"], dtype=torch.bool, device=DEV)
    touched[3, 1] = touched[sum(news) - 1, 5] = True
    assert torch.equal(out[~touched], good[~touched])


def test_views_on_two_streams_and_in_graphs():
    """Calls side by side on two streams, and two captured calls that share a workspace."""
    a = _case(64, 2, 256, 8, [4000, 900], [1, 9], 500, 4, ["any"], 16, seed=19, heavy=14)
    b = _case(32, 4, 128, 8, [600, 700], [300, 2], 130, 0, seed=20)
    want = [_run(x).clone() for x in (a, b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(5):
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(_run(x, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
    n = max(m.moe_kv_attention_workspace_bytes(x["kv"].c, x["B"], x["T"], x["H"], x["max_new"])
            for x in (a, b))
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.full_like(x["q"], 5.0) for x in (a, b)], []
    for x, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if x["tree"]:
                m.moe_kv_tree_plan(x["batch"].c, x["view"], x["B"], x["T"])
            m.moe_kv_attention_view(x["kv"].c, x["batch"].c, x["view"], x["B"], x["q"], x["T"],
                                    x["H"], x["max_new"], x["scale"], ws, n, o)
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.fill_(5.0)
            g.replay()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,kinds", [(0, None), (100, ["any"])])
def test_results_on_half_sectors(D, window, kinds):
    """`out` aligned to 16 bytes but not to 32: the same results, and nothing beside them."""
    c = _case(32, 2, D, 4, [700, 260, 33], [200, 130, 20], window, 4, kinds, 256, seed=41, heavy=14)
    good = _run(c)
    room = torch.full((c["q"].numel() + 16,), 5.0, dtype=torch.bfloat16, device=DEV)
    for at in (8, 16):
        room.fill_(5.0)
        out = room[at:at + c["q"].numel()].view(c["q"].shape)
        assert out.data_ptr() % 32 == (16 if at == 8 else 0)
        assert torch.equal(_run(c, out=out), good)
        assert torch.all(room[:at] == 5.0) and torch.all(room[at + c["q"].numel():] == 5.0)


def test_steps_without_tokens():
    """Rows without new tokens, and calls with T = 0 (whose token arrays may be missing)."""
    c = _case(16, 2, 128, 4, [30, 0, 9], [0, 0, 0], 8, 1, ["any"], 8, seed=43)
    assert torch.all(_run(c) == 5.0)
    t = c["tree"]
    for x in (t.kept, t.drop, t.last):
        x.fill_(7)
    none = dict(token=None, next_token=None, path=None)
    m.moe_kv_tree_accept(c["batch"].c, t.c, 3, 0, kept=t.kept, drop=t.drop, last=t.last, **none)
    assert [x[:3].tolist() for x in (t.kept, t.drop, t.last)] == [[0] * 3, [0] * 3, [-1] * 3]
    before = c["kv"].pool.clone()
    m.moe_kv_tree_keep(c["kv"].layers, c["batch"].c, 3, 2, t.path, t.kept)
    assert torch.equal(c["kv"].pool, before) and int(c["batch"].err[0]) == 0


@pytest.mark.parametrize("news", [[6, 2], [70, 90]])
def test_views_far_into_a_large_pool(news):
    """A pool of over 4 GB whose last blocks are in use: attention through a view, and kept tokens."""
    P, K, D, r, lens = 128, 8, 256, 2, [300, 340]
    blocks = (4 << 30) // (K * P * D * 9 // 8) + 40
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    kv = m.DeviceKv(2, 4, blocks, P, K, D)
    first = blocks - 8
    table = np.full((2, 4), -1)
    table[0, :3], table[1, :3] = blocks - 1 - np.arange(3), blocks - 4 - np.arange(3)
    kv.block_table.copy_(_ints(table))
    gen = torch.Generator(device=DEV).manual_seed(3)
    tail = kv.pool[first:]

    class Tail:
        pool = torch.empty_like(tail)

    _fill(Tail, D, gen)
    tail.copy_(Tail.pool)
    T = sum(news)
    batch = _batch(lens, news, T)
    slots = np.concatenate([table[b, np.arange(L - n, L) // P] * P + np.arange(L - n, L) % P
                            for b, (L, n) in enumerate(zip(lens, news))])
    batch.slot.copy_(_ints(slots))
    tree = m.DeviceKvTree(T, 2, max(news))
    rng = np.random.default_rng(5)
    rows = _parents(rng, news, ["bushy"], max(news))
    tree.parent.copy_(_flat(rows, T, -1))
    view = m.make_view(100, 4, tree)
    m.moe_kv_tree_plan(batch.c, view, 2, T)
    q = torch.randn(T, K * r, D, generator=gen, device=DEV).bfloat16()
    out = torch.empty_like(q)
    n = m.moe_kv_attention_workspace_bytes(kv.c, 2, T, K * r, max(news))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    m.moe_kv_attention_view(kv.c, batch.c, view, 2, q, T, K * r, max(news), D ** -0.5, ws, n, out)
    pool, start = _np(tail), 0
    for b, (L, t) in enumerate(zip(lens, news)):
        j = np.arange(L)
        k, v = ref.read_slots(pool, (table[b, j // P] - first) * P + j % P, K, P, D)
        see = tree_ref.visible(rows[b], t, L - t, 100, 4)
        qq = _f64(q[start:start + t])
        want = tree_ref.attention(qq, k, v, D ** -0.5, see)
        off = np.abs(_f64(out[start:start + t]) - want)
        assert np.all(off <= ref.attention_bound(qq, k, v, D ** -0.5, want))
        start += t
    # the last token of each row goes behind its first one
    path = [0, news[0] - 1] + [-1] * (news[0] - 2) + [0, news[1] - 1] + [-1] * (news[1] - 2)
    want = pool.copy()
    for s in (0, news[0]):
        src, dst = slots[s + news[s > 0] - 1] - first * P, slots[s + 1] - first * P
        want.reshape(-1)[_token_bytes(want, dst, K, P, D)] = pool.reshape(-1)[
            _token_bytes(want, src, K, P, D)]
    m.moe_kv_tree_keep(kv.layers, batch.c, 2, T, _ints(path), _ints([2, 2]))
    assert int(batch.err[0]) == 0
    assert np.array_equal(_np(tail), want)


# ------------------------------------------------------------------ all of them, as they are used
@pytest.mark.parametrize("P,H,K,D,rot,nodes,prompts,window,sinks", [
    (16, 8, 2, 128, 128, 12, [37, 5, 130], 24, 3),
    (64, 16, 2, 256, 64, 20, [200, 64, 1], 100, 4),
    (32, 4, 4, 64, 32, 40, [1, 31, 33], 7, 0),
])
def test_speculative_steps(P, H, K, D, rot, nodes, prompts, window, sinks):
    """Two layers, a full one and a windowed one: the prompts' chunk, then steps that draft a tree a
    row, check it and keep a path, captured once as a graph and replayed while the cache grows.  After
    each step the cache holds, in order, what was stored for the kept tokens, at their positions."""
    B, steps = len(prompts), 6
    g = torch.Generator(device=DEV).manual_seed(P + D)
    width = -(-(max(prompts) + (steps + 1) * nodes) // P)
    kv = m.DeviceKv(B, width, B * width, P, K, D, layers=2)
    rope = m.make_rope(m.rope_table(width * P, rot), rot)
    wq, wk = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    scale, windows = D ** -0.5, [(0, 0), (window, sinks)]

    def buffers(T, most, tree_max):
        s = dict(T=T, most=most, batch=m.DeviceKvBatch(T, B))
        full = m.DeviceKvTree(T, B, tree_max)
        s["trees"] = [full, m.DeviceKvTree(T, B, tree_max, parent=full.parent)]
        s["views"] = [m.make_view(w, k, t) for (w, k), t in zip(windows, s["trees"])]
        s["x"] = torch.randn(2, T, H + 2 * K, D, generator=g, device=DEV).bfloat16()
        s["q"] = torch.zeros(2, T, H, D, dtype=torch.bfloat16, device=DEV)
        s["out"] = torch.zeros_like(s["q"])
        s["new"], s["token"], s["next"] = (_ints(np.zeros(k)) for k in (B, T, T))
        s["ws"] = torch.empty(m.moe_kv_attention_workspace_bytes(kv.c, B, T, H, most),
                              dtype=torch.uint8, device=DEV)
        return s

    def step(s):
        T, batch, t = s["T"], s["batch"].c, s["trees"][0]
        m.moe_kv_plan(kv.c, s["new"], B, batch)
        for v in s["views"]:
            m.moe_kv_tree_plan(batch, v, B, T)
        for l in range(2):
            x = s["x"][l]
            proj = m.make_qkv(x[:, :H], x[:, H:H + K], x[:, H + K:], wq, wk)
            m.moe_qkv_store(kv.layers[l], batch, rope, proj, T, None, s["q"][l])
            m.moe_kv_attention_view(kv.layers[l], batch, s["views"][l], B, s["q"][l], T, H, s["most"],
                                    scale, s["ws"], s["ws"].numel(), s["out"][l])
        m.moe_kv_tree_accept(batch, t.c, B, T, s["token"], s["next"], t.path, t.kept, t.drop, t.last)

    def settle(s):
        t = s["trees"][0]
        m.moe_kv_tree_keep(kv.layers, s["batch"].c, B, s["T"], t.path, t.kept)
        m.moe_kv_plan(kv.c, t.drop, B, s["batch"].c)

    length = [0] * B
    keys = [[np.zeros((0, K, D)) for _ in range(B)] for _ in range(2)]  # the cache as it should be

    def read(l, b, L):
        j, table = np.arange(L), _np(kv.block_table)
        return ref.read_slots(_np(kv.pools[l]), table[b, j // P] * P + j % P, K, P, D)

    def check(s, news, rows, token, nxt):
        """Between a step and its settling."""
        assert int(s["batch"].err[0]) == 0
        start = 0
        held = []
        for b, n in enumerate(news):
            L = length[b] + n
            depth = tree_ref.depths(rows[b])
            for l in range(2):
                k, v = read(l, b, L)
                assert np.array_equal(k[:length[b]], keys[l][b])
                see = tree_ref.visible(rows[b], n, length[b], *windows[l])
                qq = _f64(s["q"][l][start:start + n])
                want = tree_ref.attention(qq, k, v, scale, see)
                off = np.abs(_f64(s["out"][l][start:start + n]) - want)
                assert np.all(off <= ref.attention_bound(qq, k, v, scale, want)), (l, b)
                # keys are turned by the tree's positions: within half a step of the group's range and
                # its scale's and bias' rounding to fp16 (2^-11)
                y = ref.norm_rotate(_f64(s["x"][l][start:start + n, H:H + K]), _np(wk), 1e-6,
                                    _np(rope.table_tensor), np.array([[length[b] + d for d in depth]]),
                                    rot, False, None)
                yg = y.reshape(n, K, -1, 64)
                lo, step_ = yg.min(-1, keepdims=True), (yg.max(-1) - yg.min(-1))[..., None] / 15
                tol = step_ * (0.5 + 16 * 2.0 ** -11) + np.abs(lo) * 2.0 ** -11 + 2.0 ** -18 * np.abs(yg).max()
                assert np.all(np.abs(k[length[b]:].reshape(yg.shape) - yg) <= tol)
                held.append(k[length[b]:])
            want_path, last = tree_ref.accept(rows[b], token[b], nxt[b])
            t = s["trees"][0]
            assert _np(t.path)[start:start + len(want_path)].tolist() == want_path
            assert int(t.kept[b]) == len(want_path) and int(t.last[b]) == last
            for l in range(2):
                keys[l][b] = np.concatenate((keys[l][b], held[2 * b + l][want_path]))
            length[b] += len(want_path)
            start += n

    # the prompts, one chunk: chains, kept whole
    s = buffers(sum(prompts), max(prompts), 1)
    s["new"].copy_(_ints(prompts))
    rows = [[tree_ref.CHAIN] + [0] * (n - 1) for n in prompts]
    s["trees"][0].parent.copy_(_flat(rows, s["T"], 0))
    step(s)
    check(s, prompts, rows, [[0] * n for n in prompts], [[0] * n for n in prompts])
    settle(s)
    # speculative steps, captured once
    s = buffers(B * nodes, nodes, nodes)
    tables = (kv.block_table, kv.seq_len, kv.free_list, kv.free_count)
    state = [t.clone() for t in tables]
    graphs = []
    for call in (step, settle):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(s)
        graphs.append(gr)
    for t, x in zip(tables, state):
        assert torch.equal(t, x)
    rng = np.random.default_rng(P)
    most_kept = 0
    for i in range(steps):
        news = [int(x) for x in rng.integers(1, nodes + 1, B)]
        rows = _parents(rng, news, ["bushy", "any", "line", "chain"][i % 2:], nodes)
        if i == 3:
            rows[0] = [tree_ref.CHAIN] + [0] * (news[0] - 1)
        token, nxt = _choices(rng, rows, 0.7)
        s["new"].copy_(_ints(news))
        s["trees"][0].parent.copy_(_flat(rows, s["T"], -1))
        s["token"].copy_(_flat(token, s["T"], 0))
        s["next"].copy_(_flat(nxt, s["T"], 0))
        s["x"].copy_(torch.randn(s["x"].shape, generator=g, device=DEV))
        graphs[0].replay()
        check(s, news, rows, token, nxt)
        graphs[1].replay()
        assert int(s["batch"].err[0]) == 0
        assert _np(kv.seq_len).tolist() == length
        most_kept = max(most_kept, int(s["trees"][0].kept.max()))
    assert most_kept > 2
    for l in range(2):
        for b in range(B):
            assert np.array_equal(read(l, b, length[b])[0], keys[l][b])
