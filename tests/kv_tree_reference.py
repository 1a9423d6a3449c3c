"""Plain restatement of drafted trees, windows and kept paths for the tests, one token at a time.
Shares no code with the library."""
import numpy as np

CHAIN = -2


def random_parents(rng, n, kind):
    """Parents of a row's n tokens: 'any' (each token follows any one before it), 'bushy' (one of
    the last few), 'line', 'star' (all follow the first), 'forest' (some follow the cached tokens)
    or 'chain' (marked as one, the other entries anything)."""
    if n == 0:
        return []
    if kind == "chain":
        return [CHAIN] + [int(x) for x in rng.integers(-9, 1000, n - 1)]
    p = [-1]
    for i in range(1, n):
        p.append({"any": int(rng.integers(0, i)), "bushy": int(rng.integers(max(0, i - 4), i)),
                  "line": i - 1, "star": 0, "forest": int(rng.integers(-1, i))}[kind])
    return p


def depths_and_paths(parents):
    """(depth of each token, list of each token's ancestors with itself)."""
    if parents and parents[0] == CHAIN:
        parents = list(range(-1, len(parents) - 1))
    depth, path = [], []
    for i, p in enumerate(parents):
        depth.append(depth[p] + 1 if p >= 0 else 0)
        path.append((path[p] if p >= 0 else []) + [i])
    return depth, path


def depths(parents):
    if parents and parents[0] == CHAIN:
        return list(range(len(parents)))
    depth = []
    for p in parents:
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return depth


def own_visible(parents, base, window, sinks):
    """bool [n, n]: the row's new tokens that each of them sees."""
    if parents and parents[0] == CHAIN:
        i = np.arange(len(parents))
        near = (i[None] > i[:, None] - window) | (base + i[None] < sinks) if window else True
        return (i[None] <= i[:, None]) & near
    depth, path = depths_and_paths(parents)
    see = np.zeros((len(parents), len(parents)), bool)
    for i, way in enumerate(path):
        for a in way:
            see[i, a] = window == 0 or depth[a] > depth[i] - window or base + depth[a] < sinks
    return see


def visible(parents, n, base, window, sinks):
    """bool [n, base + n]: the keys that each new token sees (parents None: a chain)."""
    if parents is None:
        parents = [CHAIN] + [0] * (n - 1)
    depth = np.array(depths(parents))
    j = np.arange(base)
    old = np.ones((n, base), bool)
    if window:
        old = (j[None] > base + depth[:, None] - window) | (j[None] < sinks)
    return np.concatenate((old, own_visible(parents, base, window, sinks)), 1)


def words_of(see, max_new):
    """The visibility as the library packs it: uint32 [n, ceil(max_new / 32)]."""
    n, words = len(see), -(-max_new // 32)
    bits = np.zeros((n, words * 32), np.uint64)
    bits[:, :see.shape[1]] = see
    return (bits.reshape(n, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)


def accept(parents, token, nxt):
    """(kept path, last choice) of one row."""
    n = len(parents)
    if n == 0:
        return [], -1
    if parents[0] == CHAIN:
        return list(range(n)), nxt[n - 1]
    path = [0]
    while True:
        kids = [c for c in range(n) if parents[c] == path[-1] and token[c] == nxt[path[-1]]]
        if not kids:
            return path, nxt[path[-1]]
        path.append(kids[0])


def attention(q, k, v, scale, see):
    """q float64 [n, H, D], k and v [L, K, D], see bool [n, L]."""
    n, H, D = q.shape
    r = H // k.shape[1]
    out = np.zeros((n, H, D))
    for h in range(H):
        x = np.where(see, q[:, h] @ k[:, h // r].T * scale, -np.inf)
        p = np.exp(x - x.max(-1, keepdims=True))
        out[:, h] = (p / p.sum(-1, keepdims=True)) @ v[:, h // r]
    return out
