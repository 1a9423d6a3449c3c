"""Checking trees of drafted tokens, and attention through a sliding window with first tokens that stay
visible, over the 4-bit paged key/value cache.

Each case is one pass of a serving program.  The plain forms below are elementary torch operations;
with `own` set the same passes go through the framework's calls.

A step gives row b of the batch n new tokens behind `base` cached ones.  They are a chain, or a tree:
parent[i] is the index (in the row) of the token that token i follows, -1 for one that follows the cached
tokens, and parents come before their children; -2 in the place of token 0's parent marks a chain whose tokens are
all kept.  Token i of depth d sits at position base + d and sees, of the cached tokens and its own ancestors,
those within its last `window` positions (0: all) and those at positions below `sinks`.

The tree's plan: for each new token int32 [1 + words], its depth, then a bit for each new token it sees.

The cache: a block holds P tokens of every kv head, head by head, as P/16 tiles of 16 tokens.
A tile of head_dim D (18 D bytes, G = D/64 groups) is
  K codes [16][D/2] | V codes [16][D/2] | K scale [16][G] | K bias [16][G] | V scale [G][16] | V bias [G][16]
with two 4-bit codes a byte (low nibble: even column) and fp16 scales and biases; the 16-byte chunk j of
code row r lies at chunk j ^ swizzle(r).  A value is scale * code + bias.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small server's step: four requests, a tree of 16 drafted tokens each
        {"name": "plan trees", "op": "plan", "rows": 4, "nodes": 16, "ragged": False, "most": 16, "window": 0, "sinks": 0},
        # a large batch of ragged trees for the windowed layers, a quarter of the rows plain chains
        {"name": "plan ragged trees", "op": "plan", "rows": 256, "nodes": 256, "ragged": True, "most": 256, "window": 100, "sinks": 4},
        # one request's tree checked: the kept path chosen and its keys and values moved into place in 8 layers
        {"name": "keep one", "op": "keep", "rows": 1, "nodes": 16, "ragged": False, "most": 16, "layers": 8, "cached": 300, "kv": 2, "dim": 256, "block": 64},
        # 64 requests with trees of up to 64 tokens, the 40 layers of the decode benchmark's model
        {"name": "keep batch", "op": "keep", "rows": 64, "nodes": 64, "ragged": True, "most": 64, "layers": 40, "cached": 200, "kv": 2, "dim": 256, "block": 64},
        # a tree of 16 tokens of one request on a short context: the latency of one check
        {"name": "tree one", "op": "attend", "rows": 1, "least": 1000, "most": 1000, "new": 16, "ragged": False, "tree": True, "window": 0, "sinks": 0, "heads": 16, "kv": 2, "dim": 256, "block": 64},
        # small trees of 16 requests in a windowed layer
        {"name": "tree in a window", "op": "attend", "rows": 16, "least": 400, "most": 5001, "new": 8, "ragged": True, "tree": True, "window": 1000, "sinks": 4, "heads": 32, "kv": 4, "dim": 128, "block": 32},
        # a batch of 32 requests with trees of up to 64 tokens, ragged contexts
        {"name": "tree batch", "op": "attend", "rows": 32, "least": 150, "most": 8191, "new": 64, "ragged": True, "tree": True, "window": 0, "sinks": 0, "heads": 32, "kv": 8, "dim": 128, "block": 64},
        # one request in a windowed layer of small heads: the latency of a decode step
        {"name": "window one", "op": "attend", "rows": 1, "least": 5000, "most": 5000, "new": 1, "ragged": False, "tree": False, "window": 128, "sinks": 4, "heads": 8, "kv": 8, "dim": 64, "block": 16},
        # the ordinary decode step of 64 requests in a windowed layer
        {"name": "window batch", "op": "attend", "rows": 64, "least": 150, "most": 8191, "new": 1, "ragged": False, "tree": False, "window": 1024, "sinks": 4, "heads": 32, "kv": 8, "dim": 128, "block": 64},
        # long contexts read through a wide window: 8 requests of about 128k tokens
        {"name": "window long", "op": "attend", "rows": 8, "least": 129000, "most": 131071, "new": 1, "ragged": False, "tree": False, "window": 32768, "sinks": 64, "heads": 16, "kv": 2, "dim": 256, "block": 64},
        # a whole prefill chunk of 8192 tokens on an empty cache
        {"name": "window prompt", "op": "attend", "rows": 1, "least": 8192, "most": 8192, "new": 8192, "ragged": False, "tree": False, "window": 1024, "sinks": 4, "heads": 16, "kv": 2, "dim": 256, "block": 64},
        # a later chunk of a long prompt: 2048 tokens on about 30000 cached ones
        {"name": "window chunk", "op": "attend", "rows": 1, "least": 32011, "most": 32011, "new": 2048, "ragged": False, "tree": False, "window": 4096, "sinks": 0, "heads": 32, "kv": 4, "dim": 128, "block": 64},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "keep", "attend", "attend", "attend", "attend"])
    window = rng.choice([0, _logint(rng, 1, 300)])
    if op == "plan":
        most = _logint(rng, 1, 256)
        return {"op": op, "rows": _logint(rng, 1, 256), "nodes": most, "ragged": rng.choice([True, False]),
                "most": rng.randint(most, 256), "window": window, "sinks": rng.choice([0, 4, 50]) if window else 0}
    block = rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    if op == "keep":
        most = _logint(rng, 1, 128)
        rows = _logint(rng, 1, min(128, 4096 // most))
        return {"op": op, "rows": rows, "nodes": most, "ragged": rng.choice([True, False]), "most": rng.randint(most, 256),
                "layers": _logint(rng, 1, 40), "cached": _logint(rng, 1, 200), "kv": min(kv, 512 // dim), "dim": dim, "block": block}
    heads = min(kv * rng.choice([1, 2, 4, 6, 8, 16]), 64 * 128 // dim // kv * kv)
    kind = rng.choice(["tree", "tree", "decode", "prompts"])
    window = _logint(rng, 1, 40000) if kind != "tree" or rng.random() < 0.4 else 0
    sinks = rng.choice([0, 1, 4, 4, 100]) if window else 0
    if kind == "prompts":
        rows = rng.choice([1, 1, 2, 5])
        most = _logint(rng, 60, min(16384, int(math.sqrt(1.0e9 / (heads * rows)))))
        return {"op": op, "rows": rows, "least": max(1, most // 3), "most": most, "new": _logint(rng, max(1, most // 4), most),
                "ragged": True, "tree": False, "window": window, "sinks": sinks, "heads": heads, "kv": kv, "dim": dim, "block": block}
    new = 1 if kind == "decode" else _logint(rng, 2, 128)
    rows = _logint(rng, 1, max(1, 128 // new))
    # the least of: the longest context, the cache's size, the scores' size
    most = _logint(rng, new, max(new, min(131072, 500_000_000 // (rows * kv * dim), 1_000_000_000 // (rows * heads * new))))
    return {"op": op, "rows": rows, "least": max(1, most // 4), "most": most, "new": new, "ragged": kind == "tree" and rng.random() < 0.7,
            "tree": kind == "tree", "window": window, "sinks": sinks, "heads": heads, "kv": kv, "dim": dim, "block": block}


def _lengths(case):
    """(tokens in the cache, this step's among them; tokens of this step) of each row."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] != "attend":
        new = [r.randint(1, case["nodes"]) if case["ragged"] else case["nodes"] for _ in range(case["rows"])]
        return [r.randint(0, case.get("cached", 5000)) + n for n in new], new
    total = [r.randint(case["least"], case["most"]) for _ in range(case["rows"])]
    total[-1] = case["most"]
    new = [min(t, r.randint(1, case["new"]) if case["ragged"] else case["new"]) for t in total]
    return total, new


def work(case):
    total, new = _lengths(case)
    T = sum(new)
    if case["op"] == "plan":
        # parents in, plans and positions out
        return {"bytes": T * (4 + 4 * (1 + -(-case["most"] // 32)) + 4) + 8 * len(new), "flops": 0}
    K, D = case["kv"], case["dim"]
    if case["op"] == "keep":
        # parents, tokens and choices in, paths out; a few kept tokens a row read and written in every layer
        kept = sum(min(n, 3) - 1 for n in new)
        return {"bytes": 16 * T + 20 * len(new) + 2 * kept * case["layers"] * K * D * 9 // 8, "flops": 0}
    H, W, S = case["heads"], case["window"], case["sinks"]
    keys = pairs = 0
    for t, n in zip(total, new):
        base = t - n
        if case["tree"]:
            # the cached tokens that a window leaves, and the tree's own (of which a token sees its path: about log n)
            cached = min(base, W + S) if W else base
            keys += cached + n
            pairs += n * (cached + 1 + int(2 * math.log(n)))
        else:
            keys += min(t, W + n + S) if W else t
            c = W + S if W else t
            full = max(0, min(n, c - base))  # tokens whose window holds everything before them
            pairs += full * base + full * (full + 1) // 2 + (n - full) * min(c, t)
    return {"bytes": keys * K * D * 9 // 8 + 4 * T * H * D, "flops": 4 * H * D * pairs}


# ------------------------------------------------------------------ the cache's layout
def _swizzle(D):
    r = torch.arange(16, device=DEV)
    return (r & 7) if D == 256 else ((r >> 1) & 3) if D == 128 else ((r >> 2) & 1)


def _chunks(D):
    """[16][D/32]: where chunk j of row r lies."""
    return torch.arange(D // 32, device=DEV)[None, :] ^ _swizzle(D)[:, None]


def _quantise(x):
    """x [..., D] float32 -> codes uint8 [..., D], scale and bias fp16 [..., G]."""
    g = x.clamp(-32768.0, 32768.0).unflatten(-1, (-1, 64))
    low = g.amin(-1)
    s = ((g.amax(-1) - low) / 15.0).half()
    b = low.half()
    sf = s.float()[..., None]
    c = torch.where(sf > 0, ((g - b.float()[..., None]) / sf), torch.zeros_like(g)).round().clamp(0, 15)
    return c.to(torch.uint8).flatten(-2), s, b


def _pack(kq, vq, D):
    """Codes, scales and biases of K and V ([N, 16, D], [N, 16, G]) -> tiles uint8 [N, 18 D]."""
    n = kq[0].shape[0]
    parts = []
    rows = torch.arange(16, device=DEV)[:, None]
    for c, _, _ in (kq, vq):
        by = (c[..., 0::2] | (c[..., 1::2] << 4)).view(n, 16, D // 32, 16)
        at = torch.empty_like(by)
        at[:, rows, _chunks(D)] = by
        parts.append(at.reshape(n, 8 * D))
    for a in (kq[1], kq[2], vq[1].transpose(1, 2), vq[2].transpose(1, 2)):
        parts.append(a.contiguous().view(torch.uint8).reshape(n, D // 2))
    return torch.cat(parts, 1)


def _unpack(tiles, D):
    """Tiles uint8 [..., 18 D] -> K and V float32 [..., 16, D]."""
    G = D // 64
    lead = tiles.shape[:-1]
    rows = torch.arange(16, device=DEV)[:, None]
    codes = tiles[..., : 16 * D].reshape(*lead, 2, 16, D // 32, 16)[..., rows, _chunks(D), :]
    codes = torch.stack((codes & 15, codes >> 4), -1).reshape(*lead, 2, 16, G, 64)
    meta = tiles[..., 16 * D:].contiguous().view(torch.float16).float()
    ks, kb = (meta[..., i * 16 * G:(i + 1) * 16 * G].reshape(*lead, 16, G, 1) for i in (0, 1))
    vs, vb = (meta[..., i * 16 * G:(i + 1) * 16 * G].reshape(*lead, G, 16).transpose(-1, -2)[..., None] for i in (2, 3))
    k = codes[..., 0, :, :, :].float() * ks + kb
    v = codes[..., 1, :, :, :].float() * vs + vb
    return k.flatten(-2), v.flatten(-2)


def _token_bytes(slot, K, D, P):
    """[T, K, D + D/8]: the bytes of a layer's pool that hold the tokens in `slot`, in an order that goes by token alone."""
    G = D // 64
    T = slot.shape[0]
    key = slot % 16
    tile = ((slot // P)[:, None] * K + torch.arange(K, device=DEV)) * (P // 16) + (slot % P // 16)[:, None]
    chunk = (_chunks(D)[key][..., None] * 16 + torch.arange(16, device=DEV)).flatten(-2)  # [T, D/2]
    code = key[:, None] * (D // 2) + chunk
    g = torch.arange(2 * G, device=DEV)
    by_key = 16 * D + key[:, None] * 2 * G + g  # K scale; its bias 32 G further
    by_group = 16 * D + 64 * G + (g // 2) * 32 + key[:, None] * 2 + g % 2  # V scale; the same
    inside = torch.cat((code, code + 8 * D, by_key, by_key + 32 * G, by_group, by_group + 32 * G), 1)
    return tile[..., None] * (18 * D) + inside.view(T, 1, -1)


# ------------------------------------------------------------------ what a program has in hand
def _state(case, rows, width, blocks, tokens, layers=1):
    """The cache and the step's buffers, by the names that a program keeps them under."""
    P, kv, dim = case.get("block", 16), case.get("kv", 1), case.get("dim", 64)
    s = {"case": dict(case), "P": P, "kv": kv, "dim": dim, "rows": rows}
    if own:
        import moe_expert_offload_gb300 as m

        s["m"] = m
        s["cache"] = m.DeviceKv(rows, width, blocks, P, kv, dim, device=DEV, layers=layers)
        s["batch"] = m.DeviceKvBatch(tokens, rows, device=DEV)
        s["stream"] = torch.cuda.current_stream().cuda_stream
        c, b = s["cache"], s["batch"]
        s.update(pools=c.pools, table=c.block_table, q_start=b.q_start, kv_len=b.kv_len, slot=b.slot, pos=b.pos)
    else:
        new = lambda n, d=torch.int32: torch.zeros(n, dtype=d, device=DEV)  # noqa: E731
        s.update(pools=[new((blocks, kv * (P // 16) * 18 * dim), torch.uint8) for _ in range(layers)], table=new((rows, width)),
                 q_start=new(rows + 1), kv_len=new(rows), slot=new(tokens), pos=new(tokens))
    return s


def _step(s, total, new, gen):
    """Blocks in random order to rows that hold `total` tokens, and the slot map of a step that brought `new` of them."""
    (rows, width), P, blocks = s["table"].shape, s["P"], s["pools"][0].shape[0]
    perm = torch.randperm(blocks, generator=gen, device=DEV).int()
    have = (torch.tensor(total, device=DEV) + P - 1) // P
    mine = torch.arange(width, device=DEV)[None, :] < have[:, None]
    rank = torch.cumsum(mine.flatten(), 0).view(rows, width) - 1
    s["table"].copy_(torch.where(mine, perm[rank.clamp(0, blocks - 1)], -1))
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    T = starts[-1]
    s["q_start"].copy_(torch.tensor(starts, device=DEV))
    s["kv_len"].copy_(torch.tensor(total, device=DEV))
    row = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV))
    index = torch.arange(T, device=DEV) - s["q_start"][row]
    at = index + (s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1]))[row]
    s["slot"].fill_(-1)
    s["pos"].zero_()
    s["slot"][:T] = (s["table"][row, at // P] * P + at % P).int()
    s["pos"][:T] = at.int()
    s["T"], s["row"], s["index"] = T, row, index


def _trees(s, gen, chains):
    """Parents of random trees (each token follows any one before it); with `chains` every fourth row is a chain."""
    i, row = s["index"], s["row"]
    parent = (torch.rand(s["T"], generator=gen, device=DEV) * i).long().clamp(max=255)
    parent = torch.where(i == 0, -1, torch.minimum(parent, i - 1))
    if chains:
        parent = torch.where((row % 4 == 3) & (i == 0), -2, parent)
    return parent.int()


def _fill_pool(s, gen):
    """Every block holds quantised keys and values: unit keys, values whose size differs from token to token."""
    D = s["dim"]
    tiles = s["pools"][0].view(-1, 18 * D)
    for a in range(0, tiles.shape[0], 16384):
        n = min(16384, tiles.shape[0] - a)
        k = torch.randn(n, 16, D, generator=gen, device=DEV)
        v = torch.randn(n, 16, D, generator=gen, device=DEV) * torch.exp(0.5 * torch.randn(n, 16, 1, generator=gen, device=DEV))
        tiles[a:a + n] = _pack(_quantise(k), _quantise(v), D)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    total, new = _lengths(case)
    P, T = case.get("block", 16), sum(new)
    width, blocks = -(-max(total) // P), sum(-(-t // P) for t in total) + 2
    if case["op"] == "plan":
        s = _state(case, len(new), width, blocks, T)
        _step(s, total, new, gen)
        parent = _trees(s, gen, True)
        s["most"], s["window"], s["sinks"] = case["most"], case["window"], case["sinks"]
        if own:
            m = s["m"]
            s["tree"] = m.DeviceKvTree(T, len(new), case["most"], device=DEV)
            s["parent"], s["seen"] = s["tree"].parent, s["tree"].seen
            s["view"] = m.make_view(window=case["window"], sinks=case["sinks"], tree=s["tree"])
            s["parent"].copy_(parent)
        else:
            s["parent"] = parent
            s["seen"] = torch.zeros(T, 1 + -(-case["most"] // 32), dtype=torch.int32, device=DEV)
        return s
    if case["op"] == "keep":
        s = _state(case, len(new), width, blocks, T, case["layers"])
        _step(s, total, new, gen)
        for p in s["pools"]:
            p.copy_(torch.randint(0, 256, p.shape, generator=gen, device=DEV, dtype=torch.uint8))
        s["parent"] = _trees(s, gen, True)
        # what the drafter proposed at each token of the tree, and what the model chooses behind it: often the proposal
        # of a child (one behind the first eight tokens, so that what is moved does not lie where something goes)
        s["token"] = torch.randint(0, 100000, (T,), generator=gen, device=DEV, dtype=torch.int32)
        start = s["q_start"].long()[s["row"]]
        depth = torch.where(s["parent"] < 0, 0, 1)
        up = torch.where(s["parent"] < 0, -1, start + s["parent"])
        for _ in range(8):
            at = up.clamp(min=0)
            depth, up = depth + torch.where(up < 0, 0, depth[at]), torch.where(up < 0, -1, up[at])
        child = torch.full((T,), T, dtype=torch.int64, device=DEV)
        t = torch.arange(T, device=DEV)
        fits = (s["parent"] >= 0) & (s["index"] >= 8) & (depth < 8)
        child.scatter_reduce_(0, torch.where(fits, start + s["parent"], t), torch.where(fits, t, T), "amin")
        takes = (child < T) & (torch.rand(T, generator=gen, device=DEV) < 0.8)
        other = torch.randint(100000, 150000, (T,), generator=gen, device=DEV, dtype=torch.int32)
        s["next"] = torch.where(takes, s["token"][child.clamp(max=T - 1)], other)
        names = ("path", T), ("kept", len(new)), ("drop", len(new)), ("last", len(new))
        if own:
            s["tree"] = s["m"].DeviceKvTree(T, len(new), case["most"], device=DEV)
            s["tree"].parent.copy_(s["parent"])
            s.update({n: getattr(s["tree"], n) for n, _ in names})
        else:
            s.update({n: torch.zeros(k, dtype=torch.int32, device=DEV) for n, k in names})
        s["most_new"] = max(new)
        return s
    H, D = case["heads"], case["dim"]
    s = _state(case, len(new), width, blocks, T)
    _step(s, total, new, gen)
    _fill_pool(s, gen)
    s["q"] = (1.5 * torch.randn(T, H, D, generator=gen, device=DEV)).bfloat16()
    s["out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    s["scale"] = D ** -0.5
    s["most_new"], s["most"], s["window"], s["sinks"] = max(new), max(total), case["window"], case["sinks"]
    s["parent"] = _trees(s, gen, True) if case["tree"] else None
    if own:
        m = s["m"]
        tree = None
        if case["tree"]:
            tree = s["tree"] = m.DeviceKvTree(T, len(new), max(new), device=DEV)
            tree.parent.copy_(s["parent"])
        s["view"] = m.make_view(window=s["window"], sinks=s["sinks"], tree=tree)
        if tree:
            m.moe_kv_tree_plan(s["batch"].c, s["view"], len(new), T, s["stream"])
        s["bytes"] = m.moe_kv_attention_workspace_bytes(s["cache"].c, len(new), T, H, max(new))
        s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    elif case["tree"]:
        s["depth"], s["sight"] = _ancestors(s, s["most_new"])
    return s


# ------------------------------------------------------------------ the passes
def run(s):
    op = s["case"]["op"]
    if op == "plan":
        return _own_plan(s) if own else _plain_plan(s)
    if op == "keep":
        return _own_keep(s) if own else _plain_keep(s)
    return _own_attend(s) if own else _plain_attend(s)


def _own_plan(s):
    s["m"].moe_kv_tree_plan(s["batch"].c, s["view"], s["rows"], s["T"], s["stream"])
    return {"seen": s["seen"], "pos": s["pos"]}


def _own_keep(s):
    m, t = s["m"], s["tree"]
    m.moe_kv_tree_accept(s["batch"].c, t.c, s["rows"], s["T"], s["token"], s["next"], t.path, t.kept, t.drop, t.last, s["stream"])
    m.moe_kv_tree_keep(s["cache"].layers, s["batch"].c, s["rows"], s["T"], t.path, t.kept, s["stream"])
    return _keep_outputs(s)


def _own_attend(s):
    s["m"].moe_kv_attention_view(s["cache"].c, s["batch"].c, s["view"], s["rows"], s["q"], s["T"], s["case"]["heads"], s["most_new"],
                                 s["scale"], s["ws"], s["bytes"], s["out"], s["stream"])
    return s["out"]


def _keep_outputs(s):
    return {**{k: s[k] for k in ("path", "kept", "drop", "last")}, "pools": s["pools"]}


def _up(s):
    """The token that each token follows, as an index of the whole batch; -1: a cached one."""
    start = s["q_start"].long()[s["row"]]
    chain = s["parent"][start] == -2
    up = torch.where(chain, s["index"] - 1, s["parent"].long())
    return torch.where(up < 0, -1, start + up), start, chain


def _ancestors(s, most):
    """depth [T]; bool [T, most]: the row's new tokens that a token sees without a window, itself and its ancestors."""
    up, start, _ = _up(s)
    depth = (up >= 0).long()
    sight = torch.arange(most, device=DEV)[None] == s["index"][:, None]
    for _ in range(max(1, (most - 1).bit_length())):  # each round reaches twice as far
        at, live = up.clamp(min=0), up >= 0
        sight = sight | (sight[at] & live[:, None])
        depth = depth + torch.where(live, depth[at], 0)
        up = torch.where(live, up[at], -1)
    return depth, sight


def _windowed(s, depth, sight, most):
    """What a window leaves of it."""
    if not s["window"]:
        return sight
    start = s["q_start"].long()[s["row"]]
    base = (s["kv_len"] - s["q_start"].diff())[s["row"]].long()
    other = (start[:, None] + torch.arange(most, device=DEV)[None]).clamp(max=s["T"] - 1)
    near = (depth[other] > depth[:, None] - s["window"]) | (base[:, None] + depth[other] < s["sinks"])
    return sight & near


def _plain_plan(s):
    most = s["most"]
    depth, sight = _ancestors(s, most)
    sight = _windowed(s, depth, sight, most)
    bits = torch.zeros(s["T"], -(-most // 32) * 32, dtype=torch.int64, device=DEV)
    bits[:, :most] = sight
    words = (bits.view(s["T"], -1, 32) << torch.arange(32, device=DEV)).sum(-1)
    s["seen"][:, 0] = depth
    s["seen"][:, 1:] = torch.where(words >= 2 ** 31, words - 2 ** 32, words)
    s["pos"].copy_((s["kv_len"] - s["q_start"].diff())[s["row"]] + depth)
    return {"seen": s["seen"], "pos": s["pos"]}


def _plain_keep(s):
    T, index, row = s["T"], s["index"], s["row"]
    up, start, chain = _up(s)
    t, at = torch.arange(T, device=DEV), up.clamp(min=0)
    # of a token's children the first one that is what the model chose
    match = (up >= 0) & (s["token"] == s["next"][at])
    first = torch.full((T + 1,), T, dtype=torch.int64, device=DEV)
    first.scatter_reduce_(0, torch.where(match, at, T), torch.where(match, t, T), "amin")
    good = chain | (index == 0) | (match & (first[at] == t))
    depth = (up >= 0).long()
    for _ in range(max(1, (s["most_new"] - 1).bit_length())):
        at, live = up.clamp(min=0), up >= 0
        good = good & (good[at] | ~live)
        depth = depth + torch.where(live, depth[at], 0)
        up = torch.where(live, up[at], -1)
    path = torch.full((T + 1,), -1, dtype=torch.int64, device=DEV)
    path.scatter_(0, torch.where(good, start + depth, T), torch.where(good, index, -1))
    path = path[:T]
    s["path"].copy_(path)
    kept = torch.zeros(s["rows"], dtype=torch.int64, device=DEV).scatter_add_(0, row, good.long())
    s["kept"].copy_(kept)
    s["drop"].copy_(kept - s["q_start"].diff())
    s["last"].copy_(s["next"][s["q_start"][:-1].long() + path[s["q_start"][:-1].long() + kept - 1]])
    slot = s["slot"].long()
    source = torch.where(path >= 0, slot[start + path.clamp(min=0)], slot)
    of, to = (_token_bytes(x, s["kv"], s["dim"], s["P"]) for x in (source, slot))
    for pool in s["pools"]:
        pool.view(-1)[to] = pool.view(-1)[of]
    return _keep_outputs(s)


def _plain_attend(s):
    D, P, K, B = s["dim"], s["P"], s["kv"], s["rows"]
    H, n, T = s["case"]["heads"], s["most_new"], s["T"]
    r, width = H // K, -(-s["most"] // P)
    table = s["table"][:, :width].long().clamp(min=0)
    tiles = s["pools"][0].view(-1, K, P // 16, 18 * D)[table]  # [B, blocks, K, P/16, 18 D]
    k, v = _unpack(tiles.permute(0, 2, 1, 3, 4).reshape(B, K, -1, 18 * D), D)
    k, v = k.flatten(2, 3), v.flatten(2, 3)  # [B, K, L, D]
    L = k.shape[2]
    row, i = s["row"], s["index"]
    q = torch.zeros(B, n, H, D, device=DEV)
    q[row, i] = s["q"].float()
    q = q.view(B, n, K, r, D).transpose(1, 2).reshape(B, K, n * r, D)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(B, K, n, r, L)
    # what token i of row b sees: [B, n, L]
    j = torch.arange(L, device=DEV)
    length, base = s["kv_len"].long(), (s["kv_len"] - s["q_start"].diff()).long()
    depth = torch.arange(n, device=DEV).expand(B, n).clone()
    hidden = j >= length[:, None, None]
    if s["parent"] is None:
        hidden = hidden | (j > (base[:, None] + depth)[..., None])
    else:
        depth[row, i] = s["depth"]
        among = torch.zeros(B, n, n, dtype=torch.bool, device=DEV)
        among[row, i] = _windowed(s, s["depth"], s["sight"], n)
        where = (j[None] - base[:, None]).clamp(0, n - 1)[:, None].expand(B, n, L)
        hidden = hidden | ((j >= base[:, None, None]) & ~among.gather(2, where))
    if s["window"]:
        far = (j <= (base[:, None] + depth)[..., None] - s["window"]) & (j >= s["sinks"])
        hidden = hidden | (far & (j < base[:, None, None]) if s["parent"] is not None else far)
    x.masked_fill_(hidden[:, None, :, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    o = torch.matmul(x.view(B, K, n * r, -1), torch.where((j[None] < length[:, None])[:, None, :, None], v, 0))
    o = o.view(B, K, n, r, D) / x.sum(-1, keepdim=True)
    s["out"].copy_(o.transpose(1, 2).reshape(B, n, H, D)[row, i])
    return s["out"]


# ------------------------------------------------------------------ in 64 bits, from the definitions
def exact(case, seed):
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    D, K, P, H = s["dim"], s["kv"], s["P"], case["heads"]
    r, W, S = H // K, case["window"], case["sinks"]
    d = torch.arange(D, device=DEV)
    total, new = _lengths(case)
    parents = s["parent"].tolist() if case["tree"] else None
    pool = s["pools"][0].view(-1)
    halves = pool.view(torch.float16)
    out = torch.empty(s["T"], H, D, dtype=torch.float64, device=DEV)
    start = 0
    for b, (L, n) in enumerate(zip(total, new)):
        base = L - n
        place, path = list(range(n)), None  # depth of each token; the new tokens on its way
        if case["tree"] and parents[start] != -2:
            path = torch.zeros(n, n, dtype=torch.bool)
            for i in range(n):
                up = parents[start + i]
                place[i] = place[up] + 1 if up >= 0 else 0
                if up >= 0:
                    path[i] = path[up]
                path[i, i] = True
            path = path.to(DEV)
        at = base + torch.tensor(place, device=DEV)  # [n] positions
        line_of = torch.cat((torch.arange(base, device=DEV), at))  # [L] positions of the row's keys
        low = max(0, base - W + 1) if W else 0  # nobody sees the keys between the sinks and this one
        keep = torch.cat((torch.arange(min(S, low), device=DEV), torch.arange(low, L, device=DEV)))
        line = keep % 16
        swizzle = {256: line % 8, 128: line // 2 % 4, 64: line // 4 % 2}[D]
        byte = line[:, None] * (D // 2) + ((d // 32)[None] ^ swizzle[:, None]) * 16 + (d % 32 // 2)[None]
        for h in range(K):
            tile = ((s["table"][b].long()[keep // P] * K + h) * (P // 16) + keep % P // 16) * (18 * D)
            kv = []
            for which in (0, 1):
                code = (pool[tile[:, None] + which * 8 * D + byte] >> (4 * (d % 2)).to(torch.uint8)[None]) % 16
                spot = (line[:, None] * (D // 64) + (d // 64)[None]) if which == 0 else ((d // 64)[None] * 16 + line[:, None])
                meta = (tile[:, None] + 16 * D + which * D) // 2 + spot
                kv.append(code.double() * halves[meta].double() + halves[meta + D // 4].double())
                del code, spot, meta
            q = s["q"][start:start + n, h * r:(h + 1) * r].double()
            for c0 in range(0, n, 1024):
                c1 = min(n, c0 + 1024)
                # the keys that these tokens may see
                some = (keep > base + c0 - W) | (keep < S) if W and path is None else torch.ones_like(keep, dtype=torch.bool)
                some = (some & (keep < base + c1)).nonzero()[:, 0]
                key = keep[some]
                mine = at[c0:c1, None]
                if path is None:
                    sees = key[None] <= mine
                else:
                    sees = (key < base)[None] | path[c0:c1][:, (key - base).clamp(min=0)]
                if W:
                    sees = sees & ((line_of[key][None] > mine - W) | (line_of[key][None] < S))
                for a in range(r):
                    x = (q[c0:c1, a] @ kv[0][some].T * s["scale"]).masked_fill(~sees, -math.inf)
                    out[start + c0:start + c1, h * r + a] = torch.softmax(x, -1) @ kv[1][some]
        start += n
    return out
