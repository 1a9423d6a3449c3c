"""The attention half of a decoder layer for serving: block tables and slot maps built on the GPU,
query/key norms with rotation stored into a 4-bit paged cache, and attention over that cache.

Each case is one pass of a serving program.  The plain forms below are elementary torch operations;
with `own` set the same passes go through the framework's calls.

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
        # a decode step of a small server: 64 requests, one new token each
        {"name": "plan decode", "op": "plan", "rows": 64, "block": 64, "cached": 8000, "new": 1, "width": 256},
        # a step that takes in prompts: 256 requests, new lengths ragged up to 1000
        {"name": "plan prompts", "op": "plan", "rows": 256, "block": 16, "cached": 2000, "new": 1000, "width": 400},
        # one decode step of 8 requests: 16 query heads on 2 kv heads of 256, a quarter of each head rotated
        {"name": "store decode", "op": "store", "tokens": 8, "heads": 16, "kv": 2, "dim": 256, "rot": 64, "pairs": "half", "axes": 1, "block": 64, "first": 20000},
        # a whole prefill chunk of 8192 tokens of the same layer
        {"name": "store prompt", "op": "store", "tokens": 8192, "heads": 16, "kv": 2, "dim": 256, "rot": 64, "pairs": "half", "axes": 1, "block": 64, "first": 0},
        # an odd chunk with image tokens: positions with three axes, whole heads of 128 rotated
        {"name": "store three axes", "op": "store", "tokens": 1237, "heads": 32, "kv": 8, "dim": 128, "rot": 128, "pairs": "adjacent", "axes": 3, "block": 16, "first": 517},
        # one request, a short context: the latency of a single decode step
        {"name": "attend one", "op": "attend", "rows": 1, "least": 1000, "most": 1000, "new": 1, "ragged": False, "heads": 16, "kv": 2, "dim": 256, "block": 64},
        # a batch of 64 requests of ragged lengths, the ordinary decode step
        {"name": "attend batch", "op": "attend", "rows": 64, "least": 150, "most": 8191, "new": 1, "ragged": False, "heads": 32, "kv": 8, "dim": 128, "block": 64},
        # long contexts: 8 requests of about 128k tokens
        {"name": "attend long", "op": "attend", "rows": 8, "least": 129000, "most": 131071, "new": 1, "ragged": False, "heads": 16, "kv": 2, "dim": 256, "block": 64},
        # checking four drafted tokens a request
        {"name": "attend drafts", "op": "attend", "rows": 16, "least": 400, "most": 5001, "new": 4, "ragged": False, "heads": 32, "kv": 4, "dim": 128, "block": 32},
        # a whole prefill chunk of 8192 tokens on an empty cache
        {"name": "attend prompt", "op": "attend", "rows": 1, "least": 8192, "most": 8192, "new": 8192, "ragged": False, "heads": 16, "kv": 2, "dim": 256, "block": 64},
        # a later chunk of a long prompt: 2048 tokens on about 30000 cached ones
        {"name": "attend chunk", "op": "attend", "rows": 1, "least": 32011, "most": 32011, "new": 2048, "ragged": False, "heads": 32, "kv": 4, "dim": 128, "block": 64},
        # seven prompts of odd lengths at once, a kv head for every query head
        {"name": "attend prompts", "op": "attend", "rows": 7, "least": 130, "most": 2001, "new": 2001, "ragged": True, "heads": 8, "kv": 8, "dim": 64, "block": 16},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "store", "attend", "attend", "attend"])
    block = rng.choice([16, 32, 64, 128])
    if op == "plan":
        new = rng.choice([1, 1, _logint(rng, 2, 1000)])
        rows = _logint(rng, 1, min(1024, 256000 // new))
        cached = _logint(rng, 1, 8000)
        return {"op": op, "rows": rows, "block": block, "cached": cached, "new": new,
                "width": -(-(cached + new) // block) + rng.randint(0, 40)}
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 6, 8, 16])
    if op == "store":
        heads = min(heads, 8192 // dim // kv * kv)
        return {"op": op, "tokens": _logint(rng, 1, 8192), "heads": heads, "kv": kv, "dim": dim,
                "rot": 16 * rng.randint(1, dim // 16), "pairs": rng.choice(["half", "adjacent"]),
                "axes": rng.choice([1, 1, 3]), "block": block, "first": _logint(rng, 1, 30000)}
    heads = min(heads, 64 * 128 // dim // kv * kv)
    kind = rng.choice(["decode", "decode", "drafts", "prompts"])
    if kind == "prompts":
        rows = rng.choice([1, 1, 2, 5])
        most = _logint(rng, 60, min(16384, int(math.sqrt(1.0e9 / (heads * rows)))))
        return {"op": op, "rows": rows, "least": max(1, most // 3), "most": most, "new": _logint(rng, max(1, most // 4), most),
                "ragged": True, "heads": heads, "kv": kv, "dim": dim, "block": block}
    rows = _logint(rng, 1, 128)
    most = _logint(rng, 1, min(131072, 500_000_000 // (rows * kv * dim)))
    new = 1 if kind == "decode" else rng.randint(1, 8)
    return {"op": op, "rows": rows, "least": max(1, most // 4), "most": most, "new": new, "ragged": kind == "drafts",
            "heads": heads, "kv": kv, "dim": dim, "block": block}


def _lengths(case):
    """(tokens in the cache, this step's among them; tokens of this step) of each row."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    total = [r.randint(case["least"], case["most"]) for _ in range(case["rows"])]
    total[-1] = case["most"]
    new = [min(t, r.randint(1, case["new"]) if case["ragged"] else case["new"]) for t in total]
    return total, new


def _plan_lengths(case):
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    old = [r.randint(0, case["cached"]) for _ in range(case["rows"])]
    new = [1 if case["new"] == 1 or r.random() < 0.25 else r.randint(1, case["new"]) for _ in old]
    return old, new


def work(case):
    if case["op"] == "plan":
        old, new = _plan_lengths(case)
        P = case["block"]
        blocks = sum(-(-(o + n) // P) - -(-o // P) for o, n in zip(old, new))
        # lengths in and out, the slots and positions, and each block taken and given back once
        return {"bytes": 2 * 20 * case["rows"] + 8 * sum(new) + 2 * 12 * blocks, "flops": 0}
    H, K, D = case["heads"], case["kv"], case["dim"]
    if case["op"] == "store":
        T = case["tokens"]
        # q, k and v in, q out, the cache's 4.5 bits a value written and read, k and v back in bf16
        return {"bytes": T * (2 * (H + 2 * K) * D + 2 * H * D + 2 * 9 * K * D // 8 + 4 * K * D + 4 * case["rot"]),
                "flops": 12 * T * (H + 2 * K) * D}
    total, new = _lengths(case)
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(total, new))
    return {"bytes": sum(total) * K * D * 9 // 8 + 4 * sum(new) * H * D, "flops": 4 * H * D * pairs}


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


# ------------------------------------------------------------------ what a program has in hand
def _state(case, gen, rows, width, blocks, kv, dim, tokens):
    """The cache and the step's buffers, by the names that a program keeps them under."""
    P = case["block"]
    s = {"case": dict(case), "P": P, "kv": kv, "dim": dim, "rows": rows}
    if own:
        import moe_expert_offload_gb300 as m

        s["m"] = m
        s["cache"] = m.DeviceKv(rows, width, blocks, P, kv, dim, device=DEV)
        s["batch"] = m.DeviceKvBatch(tokens, rows, device=DEV)
        s["stream"] = torch.cuda.current_stream().cuda_stream
        c, b = s["cache"], s["batch"]
        s.update(pool=c.pool, table=c.block_table, seq_len=c.seq_len, free=c.free_list, count=c.free_count,
                 q_start=b.q_start, kv_len=b.kv_len, slot=b.slot, pos=b.pos)
    else:
        new = lambda n, d=torch.int32: torch.zeros(n, dtype=d, device=DEV)  # noqa: E731
        s.update(pool=new((blocks, kv * (P // 16) * 18 * dim), torch.uint8), table=new((rows, width)), seq_len=new(rows),
                 free=new(blocks), count=new(1), q_start=new(rows + 1), kv_len=new(rows), slot=new(tokens), pos=new(tokens))
    return s


def _give_blocks(s, lengths, gen):
    """Blocks in random order to rows that hold `lengths` tokens; the others are free."""
    blocks, (rows, width) = s["free"].shape[0], s["table"].shape
    perm = torch.randperm(blocks, generator=gen, device=DEV).int()
    have = (torch.tensor(lengths, device=DEV) + s["P"] - 1) // s["P"]
    mine = torch.arange(width, device=DEV)[None, :] < have[:, None]
    rank = torch.cumsum(mine.flatten(), 0).view(rows, width) - 1
    s["table"].copy_(torch.where(mine, perm[rank.clamp(0, blocks - 1)], -1))
    s["seq_len"].copy_(torch.tensor(lengths, device=DEV))
    used = int(have.sum())
    s["free"].copy_(torch.roll(perm, -used))
    s["count"].fill_(blocks - used)


def _step(s, total, new):
    """The slot map of a step whose rows now hold `total` tokens, `new` of them this step's."""
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    T = starts[-1]
    s["q_start"].copy_(torch.tensor(starts, device=DEV))
    s["kv_len"].copy_(torch.tensor(total, device=DEV))
    row = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV))
    at = torch.arange(T, device=DEV) - s["q_start"][row] + (s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1]))[row]
    s["slot"].fill_(-1)
    s["pos"].zero_()
    s["slot"][:T] = (s["table"][row, at // s["P"]] * s["P"] + at % s["P"]).int()
    s["pos"][:T] = at.int()


def _fill_pool(s, gen):
    """Every block holds quantised keys and values: unit keys, values whose size differs from token to token."""
    D = s["dim"]
    tiles = s["pool"].view(-1, 18 * D)
    for a in range(0, tiles.shape[0], 16384):
        n = min(16384, tiles.shape[0] - a)
        k = torch.randn(n, 16, D, generator=gen, device=DEV)
        v = torch.randn(n, 16, D, generator=gen, device=DEV) * torch.exp(0.5 * torch.randn(n, 16, 1, generator=gen, device=DEV))
        tiles[a:a + n] = _pack(_quantise(k), _quantise(v), D)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    P = case["block"]
    if case["op"] == "plan":
        old, new = _plan_lengths(case)
        width = max(case["width"], max(-(-(o + n) // P) for o, n in zip(old, new)))
        blocks = sum(-(-(o + n) // P) for o, n in zip(old, new)) + 37
        s = _state(case, gen, len(old), width, blocks, 1, 64, sum(new) + 5)
        _give_blocks(s, old, gen)
        s["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        s["back"] = -s["new"]
        if own:
            s["batch2"] = s["m"].DeviceKvBatch(1, len(old), device=DEV)
        return s
    H, K, D = case["heads"], case["kv"], case["dim"]
    if case["op"] == "store":
        T, first, rot = case["tokens"], case["first"], case["rot"]
        total = first + T
        s = _state(case, gen, 1, -(-total // P), -(-total // P) + 3, K, D, T)
        _give_blocks(s, [total], gen)
        _step(s, [total], [T])
        # the projection's output as it comes, q, k and v of a token side by side; bounded tails, a size for each token
        qkv = torch.rand(3, T, (H + 2 * K) * D, generator=gen, device=DEV).sum(0) - 1.5
        qkv = (qkv * torch.exp(0.3 * torch.randn(T, 1, generator=gen, device=DEV))).bfloat16()
        s["q"] = qkv[:, : H * D].unflatten(1, (H, D))
        s["k"] = qkv[:, H * D:(H + K) * D].unflatten(1, (K, D))
        s["v"] = qkv[:, (H + K) * D:].unflatten(1, (K, D))
        s["qn"] = 1 + 0.05 * torch.randn(D, generator=gen, device=DEV)
        s["kn"] = 1 + 0.05 * torch.randn(D, generator=gen, device=DEV)
        angle = torch.arange(total + 1, device=DEV, dtype=torch.float64)[:, None] * (1e7 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot))[None]
        s["angles"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        axis = [(i % 3 if case["axes"] == 3 else 0) for i in range(rot // 2)]
        s["axis"] = torch.tensor(axis, device=DEV)
        # text counts on along one axis; of an image's tokens the other two axes walk over rows and columns
        t = torch.arange(T, device=DEV) + first
        s["positions"] = torch.stack([t, t // 24, t % 24][: case["axes"]]).int()
        s["q_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty(T, K, D, dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty(T, K, D, dtype=torch.bfloat16, device=DEV)
        if own:
            s["rope"] = s["m"].make_rope(s["angles"], rot, adjacent=case["pairs"] == "adjacent", axes=case["axes"], pair_axis=axis)
            s["proj"] = s["m"].make_qkv(s["q"], s["k"], s["v"], q_norm=s["qn"], k_norm=s["kn"], eps=1e-6)
        return s
    total, new = _lengths(case)
    width = -(-max(total) // P)
    T = sum(new)
    s = _state(case, gen, len(total), width, sum(-(-t // P) for t in total) + 2, K, D, T)
    _give_blocks(s, total, gen)
    _step(s, total, new)
    _fill_pool(s, gen)
    s["q"] = (1.5 * torch.randn(T, H, D, generator=gen, device=DEV)).bfloat16()
    s["out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    s["scale"] = D ** -0.5
    s["T"], s["most_new"], s["most"] = T, max(new), max(total)
    if own:
        s["bytes"] = s["m"].moe_kv_attention_workspace_bytes(s["cache"].c, len(total), T, H, max(new))
        s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ the passes
def run(s):
    op = s["case"]["op"]
    if op == "plan":
        return _own_plan(s) if own else _plain_plan(s)
    if op == "store":
        return _own_store(s) if own else _plain_store(s)
    return _own_attend(s) if own else _plain_attend(s)


def _own_plan(s):
    m, c = s["m"], s["cache"].c
    m.moe_kv_plan(c, s["new"], s["rows"], s["batch"].c, s["stream"])
    m.moe_kv_plan(c, s["back"], s["rows"], s["batch2"].c, s["stream"])
    return _plan_outputs(s)


def _own_store(s):
    m, c, T = s["m"], s["cache"].c, s["case"]["tokens"]
    m.moe_qkv_store(c, s["batch"].c, s["rope"], s["proj"], T, s["positions"], s["q_out"], s["stream"])
    m.moe_kv_load(c, s["slot"], T, s["k_out"], s["v_out"], s["batch"].err, s["stream"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_attend(s):
    s["m"].moe_kv_attention(s["cache"].c, s["batch"].c, s["rows"], s["q"], s["T"], s["case"]["heads"], s["most_new"],
                            s["scale"], s["ws"], s["bytes"], s["out"], s["stream"])
    return s["out"]


def _plan_outputs(s):
    return {k: s[k] for k in ("q_start", "kv_len", "slot", "pos", "table", "seq_len", "free", "count")}


def _plain_change(s, change, slots):
    """Rows grow by `change` tokens (or, below zero, drop that many): blocks come from the free list's
    end in the order of rows, and go back so that they come out again in that order."""
    P, table, free = s["P"], s["table"], s["free"]
    rows, width = table.shape
    n_free = free.shape[0]
    col = torch.arange(width, device=DEV)[None, :]
    old, n = s["seq_len"].long(), change.long()
    kept = (old + n.clamp(max=0)).clamp(min=0)
    grown = kept + n.clamp(min=0)
    h0, h1, h2 = ((v + P - 1) // P for v in (old, kept, grown))
    back = (col >= h1[:, None]) & (col < h0[:, None])
    count = s["count"].long() + back.sum()
    rank = torch.cumsum(back.flatten(), 0).view(rows, width) - 1
    padded = torch.cat((free, free.new_zeros(1)))
    padded.scatter_(0, torch.where(back, count - 1 - rank, n_free).flatten(), table.flatten())
    free.copy_(padded[:n_free])
    take = (col >= h1[:, None]) & (col < h2[:, None])
    rank = torch.cumsum(take.flatten(), 0).view(rows, width) - 1
    table.copy_(torch.where(take, free[(count - 1 - rank).clamp(0, n_free - 1)], torch.where(back, -1, table)))
    s["count"].copy_(count - take.sum())
    s["seq_len"].copy_(grown)
    if slots:
        s["kv_len"].copy_(grown)
        s["q_start"][1:] = torch.cumsum(n.clamp(min=0), 0)
        T = s["slot"].shape[0]
        t = torch.arange(T, device=DEV)
        row = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
        real, row = row < rows, row.clamp(max=rows - 1)
        at = t - s["q_start"][row] + kept[row]
        at = torch.where(real, at, 0)
        s["pos"].copy_(at)
        s["slot"].copy_(torch.where(real, table[row, at // P] * P + at % P, -1))


def _plain_plan(s):
    _plain_change(s, s["new"], True)
    _plain_change(s, s["back"], False)
    return _plan_outputs(s)


def _rotate(x, cos, sin, adjacent, rot):
    """x [T, h, D] with cos and sin [T, rot/2]."""
    c, n = cos[:, None], sin[:, None]
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if adjacent else r.chunk(2, -1)
    u, v = a * c - b * n, b * c + a * n
    return torch.cat((torch.stack((u, v), -1).flatten(-2) if adjacent else torch.cat((u, v), -1), rest), -1)


def _plain_store(s):
    case, D, P = s["case"], s["dim"], s["P"]
    rot, adjacent = case["rot"], case["pairs"] == "adjacent"
    p = s["positions"].long()[s["axis"]].t()  # [T, rot/2]: each pair's own axis
    pair = torch.arange(rot // 2, device=DEV)[None]
    cos, sin = s["angles"][p, pair], s["angles"][p, pair + rot // 2]
    norm = lambda x, w: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    s["q_out"].copy_(_rotate(norm(s["q"].float(), s["qn"]), cos, sin, adjacent, rot))
    k = _rotate(norm(s["k"].float(), s["kn"]), cos, sin, adjacent, rot)
    kc, ks, kb = _quantise(k)
    vc, vs, vb = _quantise(s["v"].float())
    # into the tiles of the slots
    K, T, G = s["kv"], k.shape[0], D // 64
    slot = s["slot"].long()
    tiles = s["pool"].view(-1, K, P // 16, 18 * D)
    at, key = (slot // P, slot % P // 16), slot % 16
    where = _chunks(D)[key][:, None, :, None].expand(T, K, D // 32, 16)
    block, head, tile = at[0][:, None], torch.arange(K, device=DEV)[None], at[1][:, None]
    base = ((block * K + head) * (P // 16) + tile) * 18 * D  # [T, K] byte offsets
    flat = tiles.view(-1)
    byte = torch.arange(16, device=DEV)
    put = lambda offset, c: flat.index_put_(((base[..., None, None] + offset + key[:, None, None, None] * (D // 2) + where * 16 + byte),),  # noqa: E731
                                            (c[..., 0::2] | (c[..., 1::2] << 4)).view(T, K, D // 32, 16))
    put(0, kc)
    put(8 * D, vc)
    half = s["pool"].view(-1).view(torch.float16)
    g = torch.arange(G, device=DEV)
    meta = (base[..., None] + 16 * D) // 2
    row, column = key[:, None, None] * G + g, g * 16 + key[:, None, None]
    for i, (place, a) in enumerate(((row, ks), (row, kb), (column, vs), (column, vb))):
        half.index_put_((meta + i * 16 * G + place,), a)
    # and back
    kf, vf = _unpack(tiles[at[0], :, at[1]], D)  # [T, K, 16, D]
    pick = key[:, None, None, None].expand(T, K, 1, D)
    s["k_out"].copy_(kf.gather(2, pick)[:, :, 0])
    s["v_out"].copy_(vf.gather(2, pick)[:, :, 0])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _plain_attend(s):
    D, P, K, B = s["dim"], s["P"], s["kv"], s["rows"]
    H, n, T = s["case"]["heads"], s["most_new"], s["T"]
    r, width = H // K, -(-s["most"] // P)
    table = s["table"][:, :width].long().clamp(min=0)
    tiles = s["pool"].view(-1, K, P // 16, 18 * D)[table]  # [B, blocks, K, P/16, 18 D]
    k, v = _unpack(tiles.permute(0, 2, 1, 3, 4).reshape(B, K, -1, 18 * D), D)
    k, v = k.flatten(2, 3), v.flatten(2, 3)  # [B, K, L, D]
    t = torch.arange(T, device=DEV)
    row = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    i = t - s["q_start"][row]
    q = torch.zeros(B, n, H, D, device=DEV)
    q[row, i] = s["q"].float()
    q = q.view(B, n, K, r, D).transpose(1, 2).reshape(B, K, n * r, D)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(B, K, n, r, -1)
    count = s["q_start"][1:] - s["q_start"][:-1]
    last = (s["kv_len"] - count)[:, None] + torch.arange(n, device=DEV)[None]  # [B, n] a token's own position
    last = torch.minimum(last, s["kv_len"][:, None] - 1)
    x.masked_fill_((torch.arange(x.shape[-1], device=DEV)[None, None] > last[..., None])[:, None, :, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(x.view(B, K, n * r, -1), torch.where((torch.arange(v.shape[2], device=DEV)[None] < s["kv_len"][:, None])[:, None, :, None], v, 0))
    o = o.view(B, K, n, r, D) / x.sum(-1, keepdim=True)
    s["out"].copy_(o.transpose(1, 2).reshape(B, n, H, D)[row, i])
    return s["out"]


# ------------------------------------------------------------------ in 64 bits, from the definitions
def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    D, K, P = s["dim"], s["kv"], s["P"]
    d = torch.arange(D, device=DEV)
    if case["op"] == "store":
        rot = case["rot"]

        def rotated(x, w):
            y = x.double()
            y = y / (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            out = y.clone()
            for j in range(rot // 2):
                a, b = (2 * j, 2 * j + 1) if case["pairs"] == "adjacent" else (j, j + rot // 2)
                p = s["positions"][int(j % 3) if case["axes"] == 3 else 0].long()
                c, n = s["angles"][p, j].double()[:, None], s["angles"][p, j + rot // 2].double()[:, None]
                out[..., a], out[..., b] = y[..., a] * c - y[..., b] * n, y[..., b] * c + y[..., a] * n
            return out

        def held(x):
            y = torch.empty_like(x)
            for g in range(0, D, 64):
                part = x[..., g:g + 64]
                lo, hi = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
                step, base = ((hi - lo) / 15).to(torch.float16).double(), lo.to(torch.float16).double()
                y[..., g:g + 64] = base + step * ((part - base) / step).round().clamp(0, 15)
            return y

        return {"q": rotated(s["q"], s["qn"]), "k": held(rotated(s["k"], s["kn"])), "v": held(s["v"].double())}
    H = case["heads"]
    r = H // K
    total, new = _lengths(case)
    pool = s["pool"].view(-1)
    halves = pool.view(torch.float16)
    out = torch.empty(s["T"], H, D, dtype=torch.float64, device=DEV)
    start = 0
    for b, (L, n) in enumerate(zip(total, new)):
        j = torch.arange(L, device=DEV)
        line = j % 16
        swizzle = {256: line % 8, 128: line // 2 % 4, 64: line // 4 % 2}[D]
        byte = line[:, None] * (D // 2) + ((d // 32)[None] ^ swizzle[:, None]) * 16 + (d % 32 // 2)[None]
        for h in range(K):
            tile = ((s["table"][b].long()[j // P] * K + h) * (P // 16) + j % P // 16) * (18 * D)
            kv = []
            for which in (0, 1):
                code = (pool[tile[:, None] + which * 8 * D + byte] >> (4 * (d % 2)).to(torch.uint8)[None]) % 16
                place = (line[:, None] * (D // 64) + (d // 64)[None]) if which == 0 else ((d // 64)[None] * 16 + line[:, None])
                meta = (tile[:, None] + 16 * D + which * D) // 2 + place
                kv.append(code.double() * halves[meta].double() + halves[meta + D // 4].double())
                del code, place, meta
            q = s["q"][start:start + n, h * r:(h + 1) * r].double()
            for a in range(r):
                for c0 in range(0, n, 4096):
                    c1 = min(n, c0 + 4096)
                    x = q[c0:c1, a] @ kv[0].T * s["scale"]
                    x = x.masked_fill(j[None] > (L - n + torch.arange(c0, c1, device=DEV))[:, None], -math.inf)
                    out[start + c0:start + c1, h * r + a] = torch.softmax(x, -1) @ kv[1]
        start += n
    return out
