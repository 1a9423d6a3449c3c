"""GPU tests of the 4-bit key/value cache: block plans, the rotated quantised store, slots read
back, attention, and a decode loop of all of them, against plain 64-bit restatements
(kv_reference.py)."""
import numpy as np
import pytest

import kv_reference as ref
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


# ------------------------------------------------------------------ plans
def _check_plan(kv, batch, tab, new, max_tokens):
    refused, start, length, slot, pos = tab.plan(new, max_tokens)
    B = len(new)
    m.moe_kv_plan(kv.c, _ints(new), B, batch.c)
    err = int(batch.err[0])
    assert err == (m.MOE_DERR_KV_FULL if refused else 0)
    batch.err.zero_()
    assert np.array_equal(_np(batch.q_start)[: B + 1], start)
    assert np.array_equal(_np(batch.kv_len)[:B], length)
    assert np.array_equal(_np(batch.slot), slot)
    assert np.array_equal(_np(batch.pos), pos)
    assert np.array_equal(_np(kv.block_table), tab.table)
    assert np.array_equal(_np(kv.seq_len), tab.len)
    n = int(kv.free_count[0])
    assert _np(kv.free_list)[:n].tolist() == tab.free
    return refused


@pytest.mark.parametrize("P,rows,width,blocks,max_tokens,longest,seed", [
    (16, 1, 3, 3, 40, 30, 0), (64, 7, 5, 20, 200, 90, 1), (128, 33, 4, 60, 5000, 300, 2),
    (32, 1500, 4, 3000, 9000, 12, 3), (16, 300, 40, 5000, 20011, 200, 4),
    (16, 1025, 2, 2050, 30000, 32, 5),
])
def test_plans_match_the_bookkeeping(P, rows, width, blocks, max_tokens, longest, seed):
    rng = np.random.default_rng(seed)
    kv = m.DeviceKv(rows, width, blocks, P, 1, 64, with_pool=False)
    batch = m.DeviceKvBatch(max_tokens, rows)
    tab = ref.Tables(rows, width, blocks, P)
    m.moe_kv_reset(kv.c)
    refusals = 0
    for step in range(8):
        kind = rng.integers(0, 6, rows)
        new = np.where(kind < 2, 1, np.where(kind == 2, rng.integers(0, longest + 1, rows),
                       np.where(kind == 3, -rng.integers(1, 5, rows),
                                np.where(kind == 4, 0, -(2 ** 31 - 1)))))
        if step == 5:
            new[rng.integers(0, rows)] = width * P + 1  # longer than its row
        if step == 6:
            new = np.full(rows, width * P // 2)  # more than there is room for, mostly
        if step == 7:
            new = -tab.len  # every row given up
        refusals += _check_plan(kv, batch, tab, new, max_tokens)
    assert refusals >= 1
    assert int(kv.free_count[0]) == blocks


def test_plan_of_fewer_rows_and_edges():
    """Rows behind `rows` keep what they hold; a batch filled to the last token and the last
    block; one token too many is refused whole."""
    kv = m.DeviceKv(4, 2, 6, 16, 1, 64, with_pool=False)
    batch = m.DeviceKvBatch(64, 5)
    tab = ref.Tables(4, 2, 6, 16)
    assert not _check_plan(kv, batch, tab, [16, 0, 17, 31], 64)
    kv3, len3 = _np(kv.block_table)[3].copy(), int(kv.seq_len[3])
    assert not _check_plan(kv, batch, tab, [16, 0], 64)
    assert np.array_equal(_np(kv.block_table)[3], kv3) and int(kv.seq_len[3]) == len3
    assert _check_plan(kv, batch, tab, [0, 1], 64)  # no block left
    assert not _check_plan(kv, batch, tab, [-32, 32, -17, 1], 64)
    assert not _check_plan(kv, batch, tab, [0, -32, 32, -32], 64)
    assert _check_plan(kv, batch, tab, [32, 32, 1, 0], 64)


def test_plan_of_the_longest_batch():
    """Entries up to 2^31 - 2 of a batch of 2^31 - 1 tokens."""
    n = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    kv = m.DeviceKv(2, 700, 1400, 16, 1, 64, with_pool=False)
    batch = m.DeviceKvBatch(n, 2)
    m.moe_kv_reset(kv.c)
    batch.slot.fill_(7)
    batch.pos.fill_(7)
    tab = ref.Tables(2, 700, 1400, 16)
    refused, start, length, slot, pos = tab.plan([5000, 6001], 11001)
    assert not refused
    m.moe_kv_plan(kv.c, _ints([5000, 6001]), 2, batch.c)
    assert int(batch.err[0]) == 0
    assert np.array_equal(_np(batch.slot[:11001]), slot)
    assert np.array_equal(_np(batch.pos[:11001]), pos)
    for a in range(11001, n, 1 << 28):
        assert (batch.slot[a:a + (1 << 28)] == -1).all()
        assert not batch.pos[a:a + (1 << 28)].any()


def test_plan_refuses_tables_that_are_not_its_own():
    """A free count and row lengths that together pass the pool's blocks: flagged, nothing moves."""
    kv = m.DeviceKv(2, 4, 5, 16, 1, 64, with_pool=False)
    batch = m.DeviceKvBatch(8, 2)
    kv.seq_len.fill_(64)  # claims 8 blocks of a pool of 5, with 5 free
    before = _np(kv.block_table).copy(), _np(kv.free_list).copy()
    m.moe_kv_plan(kv.c, _ints([-64, 1]), 2, batch.c)
    assert int(batch.err[0]) == m.MOE_DERR_KV_FULL | m.MOE_DERR_KV_INDEX
    assert np.array_equal(_np(kv.block_table), before[0])
    assert np.array_equal(_np(kv.free_list), before[1])
    assert int(kv.free_count[0]) == 5 and _np(batch.q_start).tolist() == [0, 0, 0]


@pytest.mark.parametrize("bad", [-1, -5, 12, 1 << 28, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("max_tokens", [40, 5000])
def test_plan_flags_block_ids_outside_the_pool(bad, max_tokens):
    """A row whose held block has an id outside the pool: its new tokens get a slot that the store
    flags and skips, padding among them nowhere, and the id is flagged again when it goes back to
    the free list and when another row takes it."""
    P, K, D = 16, 1, 64
    kv = m.DeviceKv(3, 4, 12, P, K, D)
    kv.pool.zero_()
    batch = m.DeviceKvBatch(max_tokens, 3)

    def plan(new):
        m.moe_kv_plan(kv.c, _ints(new), 3, batch.c)
        err = int(batch.err[0])
        batch.err.zero_()
        return err, _np(batch.slot)[:_np(batch.q_start)[3]]

    assert plan([10, 20, 0])[0] == 0
    kv.block_table[0, 0] = bad
    err, slots = plan([6, 1, 0])  # positions 10 .. 15 of row 0, the last ones of its bad block
    assert err == m.MOE_DERR_KV_INDEX
    assert np.array_equal(slots[:6], np.full(6, -2 ** 31))
    assert slots[6] == int(kv.block_table[1, 1]) * P + 4
    x = torch.randn(7, 3, D, device=DEV).bfloat16()
    q = torch.full((7, 1, D), 7.0, dtype=torch.bfloat16, device=DEV)
    m.moe_qkv_store(kv.c, batch.c, None, m.make_qkv(x[:, :1], x[:, 1:2], x[:, 2:]), 7, None, q)
    assert int(batch.err[0]) == m.MOE_DERR_KV_INDEX
    batch.err.zero_()
    assert torch.all(q[:6] == 7.0) and torch.equal(q[6:], x[6:, :1])
    kk, _ = ref.read_slots(_np(kv.pool), np.setdiff1d(np.arange(12 * P), slots[6:]), K, P, D)
    assert not kk.any()
    assert plan([1, 0, 0])[0] == 0  # the row's next block is a good one
    assert plan([-17, 0, 0])[0] == m.MOE_DERR_KV_INDEX
    assert bad in _np(kv.free_list).tolist()
    err, slots = plan([0, 0, 20])
    assert err == m.MOE_DERR_KV_INDEX and kv.block_table[2, :2].tolist().count(bad) == 1
    assert np.sum(slots == -2 ** 31) in (4, 16) and not np.any(slots == -1)


# ------------------------------------------------------------------ store and load
def _slots(rng, T, blocks, P):
    return _ints(rng.permutation(blocks * P)[:T])


def _store_case(T, H, K, D, P, rot, adjacent, axes, norms, seed, gap=0):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    blocks = -(-T // P) + 2
    kv = m.DeviceKv(1, blocks, blocks, P, K, D)
    kv.pool.zero_()
    batch = m.DeviceKvBatch(T, 1)
    batch.slot.copy_(_slots(rng, T, blocks, P))
    max_pos = 5000
    pos = _ints(rng.integers(0, max_pos, (axes, T)))
    if axes == 1:
        batch.pos.copy_(pos[0])
    # q, k, v slices of one buffer; `gap` columns lie between query heads
    wide = H * (D + gap) + 2 * K * D
    buf = (torch.randn(T, wide, generator=g, device=DEV) * 1.5).bfloat16()
    q = buf[:, : H * (D + gap)].unflatten(1, (H, D + gap))[..., :D]
    k = buf[:, H * (D + gap): H * (D + gap) + K * D].unflatten(1, (K, D))
    v = buf[:, H * (D + gap) + K * D:].unflatten(1, (K, D))
    w = [1 + 0.2 * torch.randn(D, generator=g, device=DEV) if n else None for n in norms]
    table = m.rope_table(max_pos, rot, 1e6) if rot else None
    axis = [i % axes for i in range(rot // 2)]
    rope = m.make_rope(table, rot, adjacent, axes, axis) if rot else None
    return dict(kv=kv, batch=batch, pos=pos, q=q, k=k, v=v, w=w, table=table, axis=axis, rope=rope,
                eps=1e-5, rot=rot, adjacent=adjacent, T=T, H=H, K=K, D=D, P=P, axes=axes)


def _run_store(c, T=None):
    q_out = torch.full((c["T"], c["H"], c["D"]), 7.0, dtype=torch.bfloat16, device=DEV)
    proj = m.make_qkv(c["q"], c["k"], c["v"], c["w"][0], c["w"][1], c["eps"])
    m.moe_qkv_store(c["kv"].c, c["batch"].c, c["rope"], proj, c["T"] if T is None else T,
                    c["pos"] if c["axes"] > 1 else None, q_out)
    return q_out


def _expected(c):
    angles = _np(c["table"]) if c["rot"] else None
    pos = _np(c["pos"])
    return [ref.norm_rotate(_f64(x), None if w is None else _np(w), c["eps"], angles, pos, c["rot"],
                            c["adjacent"], c["axis"])
            for x, w in ((c["q"], c["w"][0]), (c["k"], c["w"][1]))] + [_f64(c["v"])]


def _check_quantised(got, y, what):
    """got: the values that the cache stands for.  A code is off by at most half a step of the
    group's scale; scale and bias are rounded to fp16 (2^-11 of themselves: 15 steps of the
    scale, and the bias), and y comes from fp32 (2^-20 of the group's largest covers its sums)."""
    n = y.shape[-1] // 64
    yg = y.reshape(*y.shape[:-1], n, 64)
    lo, hi = yg.min(-1, keepdims=True), yg.max(-1, keepdims=True)
    step, big = (hi - lo) / 15, np.maximum(np.abs(lo), np.abs(hi))
    tol = 0.5 * step * (1 + 2.0 ** -11) + 2.0 ** -11 * (15 * step + np.abs(lo)) + big * 2.0 ** -20
    tol = tol + 2.0 ** -24  # an fp16 scale or bias in the subnormal range
    off = np.abs(got.reshape(yg.shape) - yg)
    assert np.all(off <= tol + 15 * 2.0 ** -25), (what, float((off - tol).max()))


@pytest.mark.parametrize("T,H,K,D,P,rot,adjacent,axes,norms,gap", [
    (1, 16, 2, 256, 64, 64, False, 1, (1, 1), 0),
    (5, 8, 8, 64, 16, 64, True, 1, (1, 1), 0),
    (33, 32, 4, 128, 32, 128, False, 1, (1, 1), 0),
    (70, 6, 1, 256, 128, 256, True, 3, (1, 0), 256),
    (17, 5, 5, 128, 16, 96, False, 3, (0, 1), 8),
    (9, 1, 1, 64, 64, 16, False, 1, (0, 0), 0),
    (300, 7, 1, 64, 128, 48, True, 4, (1, 1), 64),
    (6, 256, 1, 64, 16, 0, False, 1, (1, 1), 0),
    (40, 3, 3, 256, 16, 80, False, 1, (1, 1), 0),
    (2049, 4, 2, 128, 64, 32, False, 1, (1, 1), 0),
])
def test_store_and_load(T, H, K, D, P, rot, adjacent, axes, norms, gap):
    c = _store_case(T, H, K, D, P, rot, adjacent, axes, norms, T + D, gap)
    q_out = _run_store(c)
    yq, yk, yv = _expected(c)
    # bf16: half a step, 2^-8 of itself; the fp32 norm and rotation add 2^-20 of the pair
    pair = np.abs(yq).max(-1, keepdims=True) * 2.0 ** -20
    assert np.all(np.abs(_f64(q_out) - yq) <= np.abs(yq) * 2.0 ** -8 + pair)
    slots = _np(c["batch"].slot)
    kk, vv = ref.read_slots(_np(c["kv"].pool), slots, K, P, D)
    _check_quantised(kk, yk, "k")
    _check_quantised(vv, yv, "v")
    assert int(c["batch"].err[0]) == 0
    # read back: scale * code + bias rounded once
    k2 = torch.empty(T, K, D, dtype=torch.bfloat16, device=DEV)
    v2 = torch.empty_like(k2)
    m.moe_kv_load(c["kv"].c, c["batch"].slot, T, k2, v2)
    for got, want in ((k2, kk), (v2, vv)):
        assert np.all(np.abs(_f64(got) - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -24 * 16)
    # nothing outside the slots was written
    free = np.setdiff1d(np.arange(c["kv"].pool.shape[0] * P), slots)
    if len(free):
        k0, v0 = ref.read_slots(_np(c["kv"].pool), free, K, P, D)
        assert not k0.any() and not v0.any()


def test_store_skips_padding_and_flags_bad_tokens():
    c = _store_case(12, 4, 2, 128, 16, 64, False, 1, (1, 1), 3)
    slots = c["batch"].slot.clone()
    c["batch"].slot[4:6] = -1
    c["batch"].slot[9] = c["kv"].pool.shape[0] * 16  # one behind the last
    c["batch"].pos[10] = 5000
    c["batch"].pos[11] = -3
    q_out = _run_store(c)
    assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
    skipped = [4, 5, 9, 10, 11]
    kept = [i for i in range(12) if i not in skipped]
    assert torch.all(q_out[skipped] == 7.0) and not torch.any(q_out[kept] == 7.0)
    kk, _ = ref.read_slots(_np(c["kv"].pool), _np(slots), 2, 16, 128)
    assert not kk[skipped].any() and np.all(np.abs(kk[kept]).sum((1, 2)) > 0)
    # fewer tokens than the batch holds: the rest is left alone
    c = _store_case(12, 4, 2, 128, 16, 64, False, 1, (1, 1), 4)
    q_out = _run_store(c, T=7)
    assert torch.all(q_out[7:] == 7.0)
    kk, _ = ref.read_slots(_np(c["kv"].pool), _np(c["batch"].slot), 2, 16, 128)
    assert not kk[7:].any()
    # load: -1 and out of range leave their rows, the same slot may come twice
    s = c["batch"].slot[:7].clone()
    s[1], s[2], s[3] = -1, c["kv"].pool.shape[0] * 16, s[0]
    k2 = torch.full((7, 2, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    v2 = k2.clone()
    c["batch"].err.zero_()
    m.moe_kv_load(c["kv"].c, s, 7, k2, v2, c["batch"].err)
    assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
    assert torch.all(k2[1:3] == 9.0) and torch.equal(k2[3], k2[0]) and not torch.any(k2[4:] == 9.0)


@pytest.mark.parametrize("slot", [-2, -64, -2 ** 31])
def test_store_and_load_flag_slots_below_the_pool(slot):
    c = _store_case(3, 4, 2, 128, 16, 64, False, 1, (1, 1), 6)
    c["batch"].slot[1] = slot
    q_out = _run_store(c)
    assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
    assert torch.all(q_out[1] == 7.0) and not torch.any(q_out[[0, 2]] == 7.0)
    k = torch.full((3, 2, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    c["batch"].err.zero_()
    m.moe_kv_load(c["kv"].c, c["batch"].slot, 3, k, v, c["batch"].err)
    assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
    assert torch.all(k[1] == 9.0) and not torch.any(k[[0, 2]] == 9.0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_store_of_unusual_values(D):
    """Constant groups, zeros, subnormals, infinities, NaN, and values past the clamp."""
    c = _store_case(8, 2, 1, D, 16, 0, False, 1, (0, 0), 5)
    k = torch.zeros(8, 1, D, device=DEV)
    k[1] = 2.5
    k[2] = 1e-30
    k[3] = 3.0
    k[3, 0, 5] = float("nan")
    k[4, 0, 0], k[4, 0, 1] = float("inf"), float("-inf")
    k[5] = torch.linspace(-3e38, 3e38, D, device=DEV)
    k[6] = torch.linspace(0, 1, D, device=DEV)
    k[7] = -65504.0
    c["k"] = k.bfloat16()
    c["v"] = c["k"].flip(0).contiguous()
    _run_store(c)
    kk, vv = ref.read_slots(_np(c["kv"].pool), _np(c["batch"].slot), 1, 16, D)
    for got, x in ((kk, _f64(c["k"])), (vv, _f64(c["v"]))):
        nan = np.isnan(x).reshape(8, 1, -1, 64).any(-1, keepdims=True)
        nan = np.broadcast_to(nan, (8, 1, D // 64, 64)).reshape(8, 1, D)
        assert np.array_equal(np.isnan(got), nan)
        x = np.where(nan, 0.0, np.clip(np.where(np.isnan(x), 0.0, x), -32768, 32768))
        _check_quantised(np.where(nan, 0.0, got), x, "unusual")
    assert np.array_equal(kk[1], np.full((1, D), 2.5)) and not kk[0].any()


# ------------------------------------------------------------------ attention
def _fill(kv, D, gen, poison):
    """Random codes, scales and biases in every tile of the pool."""
    tiles = kv.pool.view(-1, 18 * D)
    n, G = tiles.shape[0], D // 64
    tiles[:, : 16 * D] = torch.randint(0, 256, (n, 16 * D), generator=gen, device=DEV,
                                       dtype=torch.uint8)
    s = 0.1 + 0.3 * torch.rand(2, n, 16 * G, generator=gen, device=DEV)
    b = -7.5 * s + 0.3 * torch.randn(2, n, 16 * G, generator=gen, device=DEV)
    if poison is not None:
        s[:], b[:] = poison, poison
    meta = torch.cat((s[0], b[0], s[1], b[1]), 1).half()
    tiles[:, 16 * D:] = meta.view(torch.uint8)


def _attend_case(P, K, D, r, lens, news, seed, poison=False, spare=3):
    """A cache of random tokens; with `poison` every slot that no token may see is NaN."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, width = len(lens), max(1, -(-max(lens) // P)) + 1
    blocks = sum(-(-n // P) for n in lens) + spare
    kv = m.DeviceKv(B, width, blocks, P, K, D)
    T = sum(news) + 2
    batch = m.DeviceKvBatch(T, B)
    order = rng.permutation(blocks)
    table = np.full((B, width), -1)
    used = 0
    for b, n in enumerate(lens):
        k = -(-n // P)
        table[b, :k] = order[used:used + k]
        used += k
    kv.block_table.copy_(_ints(table))
    batch.kv_len.copy_(_ints(lens))
    batch.q_start.copy_(_ints(np.concatenate([[0], np.cumsum(news)])))
    _fill(kv, D, gen, None)
    if poison:
        live = np.concatenate([table[b, np.arange(n) // P] * P + np.arange(n) % P
                               for b, n in enumerate(lens)] + [np.zeros(0, np.int64)]).astype(np.int64)
        mask = np.ones(blocks * P, bool)
        mask[live] = False
        # scales and biases of the dead slots: [tile][part][...]
        G = D // 64
        meta = kv.pool.view(-1, 18 * D)[:, 16 * D:].contiguous().view(torch.float16)
        dead = torch.tensor(mask, device=DEV).view(blocks, 1, P // 16, 16).expand(-1, K, -1, -1)
        dead = dead.reshape(-1, 16)
        parts = meta.view(-1, 4, 16 * G)
        by_key = dead[:, :, None].expand(-1, 16, G).reshape(-1, 16 * G)
        by_group = dead[:, None, :].expand(-1, G, 16).reshape(-1, 16 * G)
        for i in range(4):
            parts[:, i].masked_fill_(by_key if i < 2 else by_group, float("nan"))
        kv.pool.view(-1, 18 * D)[:, 16 * D:] = meta.view(torch.uint8)
    q = (torch.randn(T, K * r, D, generator=gen, device=DEV) * 1.5).bfloat16()
    return dict(kv=kv, batch=batch, q=q, T=T, H=K * r, K=K, D=D, P=P, B=B, lens=lens, news=news,
                table=table, scale=D ** -0.5, max_new=max(1, max(news)))


def _run_attend(c, q=None, ws=None, stream=None, out=None, max_new=None):
    max_new = max_new or c["max_new"]
    if out is None:
        out = torch.full_like(c["q"], 5.0)
    n = m.moe_kv_attention_workspace_bytes(c["kv"].c, c["B"], c["T"], c["H"], max_new)
    if ws is None:
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # NaN in every float
    m.moe_kv_attention(c["kv"].c, c["batch"].c, c["B"], c["q"] if q is None else q, c["T"], c["H"],
                       max_new, c["scale"], ws, n, out, stream)
    return out


def _check_attend(c, out, rows=None, q=None):
    pool, got = _np(c["kv"].pool), _f64(out)
    q = _f64(c["q"] if q is None else q)
    start, want_all, got_all = 0, [], []
    for b, (L, n) in enumerate(zip(c["lens"], c["news"])):
        if n and (rows is None or b in rows):
            j = np.arange(L)
            k, v = ref.read_slots(pool, c["table"][b, j // c["P"]] * c["P"] + j % c["P"], c["K"],
                                  c["P"], c["D"])
            qq = q[start:start + n]
            want = ref.attention(qq, k, v, c["scale"], L - n)
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


CASES = [
    # P, kv heads, D, group, lengths, new tokens
    (64, 2, 256, 8, [1000], [1]),
    (16, 1, 64, 1, [1], [1]),
    (16, 2, 128, 8, [1, 15, 16, 17, 31, 32, 33, 63, 64, 65], [1] * 10),
    (128, 1, 256, 4, [127, 128, 129, 5, 700], [1] * 5),
    (32, 8, 64, 4, [3, 0, 257, 0, 40], [1, 0, 1, 0, 1]),
    (64, 4, 128, 6, [513, 100], [1, 1]),
    (32, 2, 128, 16, [300, 33, 90], [1, 1, 1]),
    (16, 1, 256, 16, [77, 500], [1, 1]),
    (16, 1, 64, 64, [200, 9], [1, 1]),
    (64, 1, 128, 33, [130], [2]),
    (32, 4, 128, 8, [400, 4, 129, 64, 9], [4, 4, 2, 1, 3]),
    (64, 2, 256, 8, [100, 2000], [3, 8]),
    (64, 2, 256, 8, [257], [257]),
    (16, 2, 128, 8, [130], [130]),
    (64, 2, 128, 8, [640, 128], [128, 100]),
    (128, 2, 64, 1, [300, 17, 129], [300, 17, 100]),
    (16, 1, 256, 6, [333], [200]),
    (64, 1, 128, 5, [1500, 64], [70, 64]),
    (64, 2, 256, 16, [200, 900, 0, 50], [200, 1, 0, 33]),
    (32, 2, 128, 4, [3000, 40, 2100, 1], [5, 40, 300, 1]),
    (64, 8, 64, 2, [256], [256]),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("poison", [False, True])
def test_attention(i, poison):
    P, K, D, r, lens, news = CASES[i]
    c = _attend_case(P, K, D, r, lens, news, 100 + i, poison)
    out = _run_attend(c)
    assert int(c["batch"].err[0]) == 0
    _check_attend(c, out)


@pytest.mark.parametrize("K,D,r,lens,news", [
    (1, 256, 64, [500, 1, 40], [1, 1, 1]),  # single tokens of more queries than a decode unit takes
    (1, 256, 33, [300, 17], [1, 1]),
    (2, 256, 32, [129, 700], [1, 1]),
    (1, 256, 48, [260, 16], [3, 16]),
    (2, 256, 8, [90, 1200, 33], [4, 5, 1]),  # 32 and 40 queries per kv head
    (1, 128, 64, [300, 4], [1, 2]),
    (1, 64, 63, [200, 1], [2, 1]),
])
def test_attention_where_the_kernels_meet(K, D, r, lens, news):
    c = _attend_case(32, K, D, r, lens, news, 60 + D + r, poison=True)
    out = _run_attend(c)
    assert int(c["batch"].err[0]) == 0
    _check_attend(c, out)


def test_attention_is_repeatable_and_ignores_its_workspace():
    c = _attend_case(64, 2, 128, 8, [3000, 5, 777, 1200], [1, 2, 200, 1], 7)
    first = _run_attend(c)
    for fill in (0, 1, 255):
        n = m.moe_kv_attention_workspace_bytes(c["kv"].c, c["B"], c["T"], c["H"], c["max_new"])
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(_run_attend(c, ws=ws).view(torch.int16), first.view(torch.int16))
    # a larger bound on the new tokens changes nothing but roundings
    wider = _run_attend(c, max_new=1000)
    _check_attend(c, wider)


@pytest.mark.parametrize("D,news", [(128, [1, 1, 1]), (256, [1, 1, 1]), (64, [40, 200, 3]),
                                    (256, [130, 1, 3])])
def test_attention_of_extreme_scores(D, news):
    """Queries so large that one key takes all the weight, zero queries (plain means), and
    scores that all lie far below zero."""
    c = _attend_case(32, 1, D, 8, [500, 260, 33], news, 11)
    big = c["q"].float() * 200
    big[0] = 0
    big[:, 1::3] = 0
    big[:, 2::3] = -big[:, 2::3].abs()
    q = big.bfloat16()
    out = _run_attend(c, q=q)
    # the bound's score term assumes scores of ordinary size: with weights that jump between
    # keys only finiteness, zero queries and the hull of the values are checked here
    got = _f64(out)[: sum(news)]
    assert np.all(np.isfinite(got))
    pool, start = _np(c["kv"].pool), 0
    for b, (L, n) in enumerate(zip(c["lens"], news)):
        j = np.arange(L)
        k, v = ref.read_slots(pool, c["table"][b, j // 32] * 32 + j % 32, 1, 32, D)
        lo, hi = v.min(0), v.max(0)
        slack = np.abs(v).max() * 2.0 ** -7
        g = got[start:start + n]
        assert np.all(g >= lo - slack) and np.all(g <= hi + slack)
        qz = np.zeros((n, 8, D))
        want = ref.attention(qz, k, v, 1.0, L - n)
        tol = ref.attention_bound(qz, k, v, 1.0, want)
        zero = ~_f64(q)[start:start + n].any(-1)
        assert zero.any()
        assert np.all(np.abs(g - want)[zero] <= tol[zero])
        start += n


FAR = [(D, n) for D in (256, 128, 64) for n in ([130, 260, 33], [1, 4, 2])]  # head_dim, new tokens


@pytest.mark.parametrize("size", [1e2, 1e4, 3e6, 1e9, 1e12, 1e30])
@pytest.mark.parametrize("below", [False, True])
@pytest.mark.parametrize("D,news", FAR)
def test_attention_of_far_scores(D, news, below, size):
    """Scores up to 2^100 from zero, on both sides or all below it: the result is the top key's
    value wherever no other key comes near.

    How near: a key may be formed in fp16 (2^-11 of scale * code and of the bias, and of their
    sum) and D products are summed in fp32 (2^-24 of them per addition), so a score is off by at
    most 2^-9 of the sum of its products' sizes.  Where two scores keep 2^-8 of it and 40 (of
    log2) apart, the others' weights are below L 2^-40 in all.  What is left is a value formed in
    fp16 (once, on terms of up to twice its group's largest), its weight and its product with a
    scale (2^-11 each), and the result's rounding to bf16."""
    lens, P, r = [500, 260, 33], 32, 8
    c = _attend_case(P, 1, D, r, lens, news, 31)
    q = c["q"].float() * size
    if below:  # keys about 6 above zero, queries below it
        meta = c["kv"].pool.view(-1, 18 * D)[:, 16 * D:].view(torch.float16).view(-1, 4, D // 4)
        meta[:, 1] += 6
        q = -q.abs()
    q = q.bfloat16()
    out = _run_attend(c, q=q)
    assert int(c["batch"].err[0]) == 0
    got, pool, start, checked = _f64(out), _np(c["kv"].pool), 0, 0
    assert np.all(np.isfinite(got[:sum(news)]))
    for b, (L, n) in enumerate(zip(lens, news)):
        j = np.arange(L)
        k, v = (x[:, 0] for x in ref.read_slots(pool, c["table"][b, j // P] * P + j % P, 1, P, D))
        qq = _f64(q)[start:start + n]
        seen = (j[None] <= L - n + np.arange(n)[:, None])[:, None]  # [n, 1, L]
        x = np.where(seen, qq @ k.T, -np.inf) * (c["scale"] * np.log2(np.e))
        reach = np.where(seen, np.abs(qq) @ np.abs(k).T, 0).max(-1) * (c["scale"] * 1.5)
        order = np.sort(x, -1)
        clear = order[..., -1] - (order[..., -2] if L > 1 else -np.inf) > reach * 2.0 ** -8 + 40
        clear |= seen.sum(-1) == 1
        want = v[x.argmax(-1)]
        big = np.abs(v).max(0).reshape(-1, 64).max(-1).repeat(64)
        tol = np.abs(want) * 2.0 ** -8 + 2 * big * 3 * 2.0 ** -11
        off = np.abs(got[start:start + n] - want)
        assert np.all((off <= tol)[clear]), (b, float((off - tol)[clear].max()))
        checked += int(clear.sum())
        start += n
    if size >= 1e4 and not below:
        assert checked > sum(news) * r // 2


@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4, 1e-5, "up", "down"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,n", [(256, 1), (100, 4), (16, 130)])
def test_attention_of_small_values_under_one_large_weight(B, n, D, size):
    """The first key outweighs each of the others by 2^9 to 2^13, and all of them together do not
    fall far behind it; values of one size from 1 down to where their scales are subnormal, or of
    sizes that grow (shrink) along the row.  Rows enough that one warp meets both kinds of keys.

    Scores are exact here (keys are a bias alone; 2^-20 of them for the sums and the factor, on 9
    at most), so a weight is off by 2^-11 for itself and 2^-11 for its product with a scale, a
    value formed in fp16 by 2^-11, the fp32 sums by below 2^-11 of the same terms, the score by
    2^-16; all of them act on scale * code and on the bias.  Below fp16's normal range a product
    is off by 2^-25, where the largest weight is 2^7 and the largest scale was moved to 2^-3 or
    more: 2^-29 of the largest weight and scale a key, times a code."""
    L, K, r = 1000, 8, 4
    c = _attend_case(16, K, D, r, [L] * B, [n] * B, 33)
    c["kv"].block_table[:] = c["kv"].block_table[0].clone()  # all rows read one context
    blocks, G = c["table"][0, :-(-L // 16)], D // 64
    meta = c["kv"].pool.view(-1, 18 * D)[:, 16 * D:].view(torch.float16).view(-1, K, 4, 16 * G)
    meta[:, :, :2] = 0
    meta[int(blocks[0]), :, 1, :G] = 13 * np.log(2) / D ** 0.5  # the first key of every head
    if isinstance(size, str):
        e = -16 + 24 * torch.arange(len(blocks), device=DEV) / len(blocks)
        s = torch.exp2(e if size == "up" else e.flip(0))[:, None, None].expand(-1, K, 16 * G)
    else:
        s = torch.full((len(blocks), K, 16 * G), size / 7.5, device=DEV)
    s = s.half()
    at = torch.tensor(blocks, device=DEV)
    meta[at, :, 2], meta[at, :, 3] = s, -7 * s
    q = torch.ones_like(c["q"])
    for h in range(c["H"]):
        q[:, h] = (9 + h % r * 4 / 3) / 13
    out = _run_attend(c, q=q)
    assert int(c["batch"].err[0]) == 0
    j = np.arange(L)
    k, v = ref.read_slots(_np(c["kv"].pool), blocks[j // 16] * 16 + j % 16, K, 16, D)
    qq = _f64(q)[:n]
    want = ref.attention(qq, k, v, c["scale"], L - n)
    step = _f64(s)[j // 16, 0, 0][:, None, None]
    terms = ref.attention(qq, k, np.abs(v + 7 * step) + 7 * step, c["scale"], L - n)
    tol = (np.abs(want) * 2.0 ** -8 + terms * (4 * 2.0 ** -11 + 2.0 ** -15)
           + L * 15 * step.max() * 2.0 ** -29)
    off = np.abs(_f64(out)[:B * n].reshape(B, n, -1, D) - want)
    assert np.all(off <= tol), (float((off / tol).max()), float(off.max()))


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-20, 1e-12, 1e38])
@pytest.mark.parametrize("D,news", [(64, [1, 2, 1]), (128, [1, 4, 1]), (256, [1, 2, 1]),
                                    (64, [140, 260, 33]), (128, [140, 260, 33]), (256, [140, 260, 33])])
def test_attention_with_scales_at_the_ends(D, news, scale):
    """A scale that takes the scores to nothing leaves the mean of what a token sees; a zero query
    has that of any scale, and a large one with a large query no NaN."""
    c = _attend_case(32, 1, D, 8, [500, 260, 33], news, 34)
    c["scale"] = scale
    q = c["q"].clone()
    q[:, ::2] = 0
    if scale > 1:
        q[:, 1::4] = (q[:, 1::4].float() * 1e30).bfloat16()
    out = _run_attend(c, q=q)
    assert int(c["batch"].err[0]) == 0
    got, pool, start = _f64(out)[:sum(news)], _np(c["kv"].pool), 0
    assert np.all(np.isfinite(got))
    zero = np.arange(8) % 2 == 0 if scale > 1 else np.ones(8, bool)
    for b, (L, n) in enumerate(zip(c["lens"], news)):
        j = np.arange(L)
        k, v = ref.read_slots(pool, c["table"][b, j // 32] * 32 + j % 32, 1, 32, D)
        qz = np.zeros((n, 8, D))
        want = ref.attention(qz, k, v, 1.0, L - n)
        tol = ref.attention_bound(qz, k, v, 1.0, want)
        assert np.all((np.abs(got[start:start + n] - want) <= tol)[:, zero]), b
        start += n


@pytest.mark.parametrize("scale", [1e4, 1e10, 1e30, 1e38])
@pytest.mark.parametrize("D,news", [(D, n) for D in (64, 128, 256) for n in ([1, 2, 1], [130, 260, 33])])
def test_attention_of_scores_below_fp32(D, news, scale):
    """Scores that all lie below fp32's range, queries of 1e35 against keys of one value each (the
    same in every column, so a raw score is exact but for its sum's 2^-16): the key nearest to zero
    takes all the weight, a token's only key too.  Keys differ by 2^-8 of themselves at least."""
    lens, P = [500, 260, 33], 32
    c = _attend_case(P, 1, D, 8, lens, news, 36)
    c["scale"] = scale
    G = D // 64
    meta = c["kv"].pool.view(-1, 18 * D)[:, 16 * D:].view(torch.float16).view(-1, 4, 16 * G)
    key = torch.zeros(meta.shape[0], 16)
    rng = np.random.default_rng(37)
    near = []
    for b, L in enumerate(lens):
        j = np.arange(L)
        size = 1 + rng.permutation(L) / 128  # one value a key
        tile = c["table"][b, j // P] * (P // 16) + j % P // 16
        key[tile, j % 16] = torch.tensor(size, dtype=torch.float32)
        near.append(size)
    meta[:, 0] = 0
    meta[:, 1] = key.repeat_interleave(G, 1).half().to(DEV)
    q = torch.full_like(c["q"], -1e35)
    out = _run_attend(c, q=q)
    assert int(c["batch"].err[0]) == 0
    got, pool, start = _f64(out), _np(c["kv"].pool), 0
    for b, (L, n) in enumerate(zip(lens, news)):
        j = np.arange(L)
        _, v = ref.read_slots(pool, c["table"][b, j // P] * P + j % P, 1, P, D)
        top = np.array([near[b][:L - n + i + 1].argmin() for i in range(n)])
        want = v[top, 0][:, None]
        big = np.abs(v).max((0, 1)).reshape(-1, 64).max(-1).repeat(64)
        tol = np.abs(want) * 2.0 ** -8 + 2 * big * 3 * 2.0 ** -11
        assert np.all(np.abs(got[start:start + n] - want) <= tol), b
        start += n


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news", [[1, 1], [1, 150]])
def test_attention_of_values_of_all_sizes(D, news):
    """Scales from 2^-9 to 2^9 within a row, tiny and large queries: the fp16 products keep
    their range."""
    c = _attend_case(16, 2, D, 4, [300, 200], news, 13)
    G = D // 64
    meta = c["kv"].pool.view(-1, 18 * D)[:, 16 * D:].contiguous().view(torch.float16).view(-1, 4, 16 * G)
    g = torch.Generator(device=DEV).manual_seed(1)
    f = torch.exp2(torch.randint(-9, 10, (meta.shape[0], 16 * G), generator=g, device=DEV).float())
    meta[:, 2] = (meta[:, 2].float() * f).half()
    meta[:, 3] = (meta[:, 3].float() * f).half()
    c["kv"].pool.view(-1, 18 * D)[:, 16 * D:] = meta.reshape(-1, 64 * G).view(torch.uint8)
    size = torch.exp2(torch.randint(-40, 2, (c["T"], 1, 1), generator=g, device=DEV).float())
    c["q"] = (c["q"].float() * size).bfloat16()
    _check_attend(c, _run_attend(c))


@pytest.mark.parametrize("lens,news", [([300, 70, 200], [1, 1, 1]), ([300, 260, 200], [150, 9, 130]),
                                       ([300, 260, 200], [150, 90, 130])])
def test_attention_leaves_out_bad_blocks_and_rows(lens, news):
    """Block ids outside the pool and rows whose bounds do not fit are flagged; the others'
    results stay."""
    c = _attend_case(16, 2, 128, 4, lens, news, 17)
    good = _run_attend(c)
    bad = c["kv"].block_table.clone()
    bad[1, 2] = c["kv"].pool.shape[0]
    bad[1, 0] = -1
    c["kv"].block_table.copy_(bad)
    out = _run_attend(c)
    assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
    _check_attend(c, out, rows=(0, 2))
    assert torch.all(torch.isfinite(out.float()))
    first = news[0]
    assert torch.equal(out[:first], good[:first])
    # a row without a single good block is 0
    c["kv"].block_table[1].fill_(-1)
    out = _run_attend(c)
    assert not torch.any(out[first:first + news[1]])
    # bounds: longer than the block table, more new tokens than the cache holds
    c["kv"].block_table.copy_(bad)
    for value in (c["kv"].c.max_blocks * 16 + 1, -1, news[1] - 1):
        c["batch"].err.zero_()
        c["batch"].kv_len[1] = value
        out = _run_attend(c)
        assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
        assert torch.all(out[first:first + news[1]] == 5.0)
        _check_attend(c, out, rows=(0, 2))
    c["batch"].kv_len[1] = lens[1]
    c["batch"].q_start[3] = c["T"] + 1  # past the queries
    c["batch"].err.zero_()
    out = _run_attend(c)
    assert int(c["batch"].err[0]) & m.MOE_DERR_KV_INDEX
    assert torch.all(out[sum(news[:2]):] == 5.0)


def test_attention_on_two_streams_at_once():
    a = _attend_case(64, 2, 256, 8, [4000, 900], [1, 1], 19)
    b = _attend_case(32, 4, 128, 8, [600, 700], [300, 2], 20)
    want = [_run_attend(x).clone() for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(_run_attend(x, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])


def test_attention_of_many_rows():
    """More rows than the kernels' scans take at a time, most of them short, some idle, two long
    ones among them; decode and prompt rows in one call."""
    rng = np.random.default_rng(23)
    B = 1000
    lens = rng.integers(0, 40, B)
    lens[17], lens[901], lens[999] = 700, 300, 1
    news = np.minimum(lens, rng.integers(0, 3, B))
    news[901], news[999] = 100, 1
    c = _attend_case(16, 1, 64, 4, lens.tolist(), news.tolist(), 24, poison=True)
    out = _run_attend(c)
    assert int(c["batch"].err[0]) == 0
    _check_attend(c, out)


@pytest.mark.parametrize("B", [31, 32, 33, 200, 300, 600])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_of_row_counts(B, D):
    """Around the row counts where the shares are found in another way: decode rows, idle ones and
    prompts among them, the last row a prompt."""
    rng = np.random.default_rng(B + D)
    lens = rng.integers(0, 90, B)
    news = np.minimum(lens, rng.integers(0, 3, B))
    lens[B // 2], news[B // 2] = 400, 130
    lens[B - 1], news[B - 1] = 140, 140
    c = _attend_case(16, 1, D, 4, lens.tolist(), news.tolist(), 70 + B, poison=True)
    out = _run_attend(c)
    assert int(c["batch"].err[0]) == 0
    _check_attend(c, out)


def test_attention_without_work():
    c = _attend_case(16, 2, 128, 4, [30, 0, 9], [1, 0, 1], 25)
    c["batch"].q_start.zero_()
    out = _run_attend(c)
    assert int(c["batch"].err[0]) == 0 and torch.all(out == 5.0)
    out = _run_attend(c, max_new=500)
    assert int(c["batch"].err[0]) == 0 and torch.all(out == 5.0)


@pytest.mark.parametrize("max_new", [1, 3, 100])
def test_attention_flags_rows_past_max_new(max_new):
    lens, news = [50, 300, 41, 200], [1, 150, 1, 4]
    c = _attend_case(16, 1, 128, 4, lens, news, 26)
    out = _run_attend(c, max_new=max_new)
    assert int(c["batch"].err[0]) == m.MOE_DERR_KV_INDEX
    start = 0
    for b, n in enumerate(news):
        if n > max_new:
            assert torch.all(out[start:start + n] == 5.0)
        start += n
    _check_attend(c, out, rows=[b for b, n in enumerate(news) if n <= max_new])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,news", [(64, [1, 1, 2]), (128, [1, 200, 100]), (256, [1, 3, 100])])
def test_attention_of_broken_values_stays_in_its_row(D, news, bad):
    """A value's scale that is NaN or infinite spoils the row that holds it and no other."""
    c = _attend_case(16, 2, D, 4, [250, 300, 120], news, 29)
    meta = c["kv"].pool.view(-1, 18 * D)[:, 16 * D:].view(torch.float16)  # [tile][part][...]
    G = D // 64
    block = int(c["table"][0, 3])  # row 0's tokens 48 .. 63, kv head 1
    meta[block * 2 + 1, 2 * 16 * G + 5] = bad  # V scale of group 0, token 53
    out = _run_attend(c)
    assert int(c["batch"].err[0]) == 0
    _check_attend(c, out, rows=[1, 2])
    heads = out[:news[0]].float()
    assert not torch.isfinite(heads[:, 4:, :64]).all()
    assert torch.isfinite(heads[:, :4]).all()


@pytest.mark.parametrize("news", [[1, 1], [4, 120]])
def test_attention_of_broken_queries_stays_in_its_rows(news):
    """An infinite or NaN query spoils its own output row and no other."""
    c = _attend_case(16, 2, 256, 4, [200, 300], news, 27)
    good = _run_attend(c)
    q = c["q"].clone()
    q[0, 1, 7] = float("nan")
    q[sum(news) - 1, 5, 0] = float("inf")
    out = _run_attend(c, q=q)
    touched = torch.zeros(c["T"], c["H"], dtype=torch.bool, device=DEV)
    touched[0, 1] = touched[sum(news) - 1, 5] = True
    assert torch.equal(out[~touched], good[~touched])
    assert torch.all(torch.isnan(out[0, 1].float()))


@pytest.mark.parametrize("news", [[1, 2], [70, 1]])
def test_far_blocks_of_a_large_pool(news):
    """A pool of over 4 GB whose last blocks are in use: store, load and attention."""
    P, K, D, r = 128, 8, 256, 2
    blocks = (4 << 30) // (K * P * D * 9 // 8) + 40
    kv = m.DeviceKv(2, 4, blocks, P, K, D)
    lens = [300, 140]
    batch = m.DeviceKvBatch(sum(lens), 2)
    g = torch.Generator(device=DEV).manual_seed(3)
    # the cache was filled from the low blocks up: these rows get the last ones
    kv.free_list.copy_(torch.arange(blocks, dtype=torch.int32, device=DEV))
    m.moe_kv_plan(kv.c, _ints(lens), 2, batch.c)
    assert int(batch.slot.min()) > (blocks - 6) * P
    x = torch.randn(sum(lens), K * r + 2 * K, D, generator=g, device=DEV).bfloat16()
    q = torch.empty(sum(lens), K * r, D, dtype=torch.bfloat16, device=DEV)
    proj = m.make_qkv(x[:, :K * r], x[:, K * r:K * r + K], x[:, K * r + K:])
    m.moe_qkv_store(kv.c, batch.c, None, proj, sum(lens), None, q)
    assert torch.equal(q, x[:, :K * r])
    k, v = (torch.empty(sum(lens), K, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    m.moe_kv_load(kv.c, batch.slot, sum(lens), k, v)
    table = _np(kv.block_table)
    first = int(table[table >= 0].min())
    tail = _np(kv.pool[first:])
    step = m.DeviceKvBatch(sum(news), 2)
    step.q_start.copy_(_ints([0, news[0], sum(news)]))
    step.kv_len.copy_(_ints(lens))
    qq = (torch.randn(sum(news), K * r, D, generator=g, device=DEV)).bfloat16()
    out = torch.empty_like(qq)
    n = m.moe_kv_attention_workspace_bytes(kv.c, 2, sum(news), K * r, max(news))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    m.moe_kv_attention(kv.c, step.c, 2, qq, sum(news), K * r, max(news), D ** -0.5, ws, n, out)
    assert int(step.err[0]) == 0 and int(batch.err[0]) == 0
    start = 0
    for b, (L, t) in enumerate(zip(lens, news)):
        j = np.arange(L)
        slots = (table[b, j // P] - first) * P + j % P
        kk, vv = ref.read_slots(tail, slots, K, P, D)
        at = sum(lens[:b])
        for got, want in ((k, kk), (v, vv)):
            assert np.all(np.abs(_f64(got[at:at + L]) - want) <= np.abs(want) * 2.0 ** -8)
        _check_quantised(kk, _f64(x[at:at + L, K * r:K * r + K]), "k")
        want = ref.attention(_f64(qq[start:start + t]), kk, vv, D ** -0.5, L - t)
        tol = ref.attention_bound(_f64(qq[start:start + t]), kk, vv, D ** -0.5, want)
        assert np.all(np.abs(_f64(out[start:start + t]) - want) <= tol)
        start += t


def _long_case(P, K, D, r, lens, news, cycle, climb, seed):
    """Rows that all read one context, whose blocks come again after `cycle` of them, so that long
    contexts need a small pool.  climb: the scores rise by about so much (log2) along the cycle."""
    c = _attend_case(P, K, D, r, [cycle * P] + [1] * (len(lens) - 1), news, seed)
    order = c["table"][0, :cycle]
    width = -(-max(lens) // P)
    c["table"] = np.tile(order[np.arange(width) % cycle], (len(lens), 1))
    kv = c["kv"]
    kv.block_table = _ints(c["table"])
    kv.c.block_table, kv.c.max_blocks = kv.block_table.data_ptr(), width
    c["lens"] = lens
    c["batch"].kv_len.copy_(_ints(lens))
    if climb:  # every query has a part along the ones, and a key's part along them rises
        c["q"] += 0.5
        up = climb * np.log(2) / (0.5 * D ** 0.5) * torch.arange(cycle, device=DEV) / cycle
        meta = kv.pool.view(-1, 18 * D)[:, 16 * D:].view(torch.float16).view(-1, K * P // 16, 4, D // 4)
        meta[torch.tensor(order, device=DEV), :, 1] += up.half()[:, None, None]
    return c


def _check_long(c, out):
    """_check_attend in 64 bits on the GPU, of a context that all rows share."""
    P, K, D, r = c["P"], c["K"], c["D"], c["H"] // c["K"]
    slots = np.arange(c["kv"].pool.shape[0] * P)
    k_all, v_all = (torch.tensor(x, device=DEV) for x in
                    ref.read_slots(_np(c["kv"].pool), slots, K, P, D))
    j = torch.arange(max(c["lens"]), device=DEV)
    at = torch.tensor(c["table"][0], device=DEV)[j // P] * P + j % P
    big = v_all.abs().amax(0).view(K, -1, 64).amax(-1).repeat_interleave(64, 1)  # [K, D]
    start, wrong, size = 0, 0.0, 0.0
    for L, n in zip(c["lens"], c["news"]):
        seen = j[None, :L] <= L - n + torch.arange(n, device=DEV)[:, None]
        for h in range(K):
            k, v = k_all[at[:L], h], v_all[at[:L], h]
            q = c["q"][start:start + n, h * r:(h + 1) * r].double()  # [n, r, D]
            x = (q @ k.T * c["scale"]).masked_fill(~seen[:, None], -np.inf)
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


@pytest.mark.parametrize("climb", [0, 60])
@pytest.mark.parametrize("P,K,D,r,B,least,most,n,cycle", [
    # key tiles of a warp (its share of all units' tiles): 55, 107, 54, 61
    (64, 8, 128, 4, 64, 150, 8191, 1, 128),
    (16, 2, 256, 8, 8, 129000, 131071, 1, 300),
    (32, 4, 64, 3, 40, 4000, 9000, 3, 282),
    (128, 2, 128, 16, 12, 20000, 30001, 2, 40),
    # key blocks of a CTA (128 keys): 75, 105, 74
    (64, 2, 256, 8, 2, 9000, 9400, 600, 148),
    (64, 4, 128, 8, 1, 13001, 13001, 1200, 210),
    (16, 8, 64, 1, 5, 8000, 9000, 1000, 563),
])
def test_attention_of_long_shares(P, K, D, r, B, least, most, n, cycle, climb):
    """Work enough that every warp (CTA) turns its buffers many times over, moves its means and its
    window of the block table, and cuts few units: long contexts, with references that keep
    growing on the way too."""
    rng = np.random.default_rng(P + D)
    lens = rng.integers(least, most + 1, B).tolist()
    c = _long_case(P, K, D, r, lens, [n] * B, cycle, climb, 35)
    out = _run_attend(c)
    assert int(c["batch"].err[0]) == 0
    _check_long(c, out)
    assert torch.equal(_run_attend(c), out)


def test_two_graphs_share_a_workspace():
    """Two captured calls of different shapes over one workspace, replayed one after the other."""
    a = _attend_case(64, 2, 128, 8, [900, 30], [1, 1], 28)
    b = _attend_case(16, 2, 128, 8, [400, 200], [300, 2], 29)
    want = [_run_attend(x).clone() for x in (a, b)]
    n = max(m.moe_kv_attention_workspace_bytes(x["kv"].c, x["B"], x["T"], x["H"], x["max_new"])
            for x in (a, b))
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.full_like(x["q"], 5.0) for x in (a, b)], []
    for x, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_kv_attention(x["kv"].c, x["batch"].c, x["B"], x["q"], x["T"], x["H"], x["max_new"],
                               x["scale"], ws, n, o)
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.fill_(5.0)
            g.replay()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


# ------------------------------------------------------------------ all of them, as they are used
@pytest.mark.parametrize("P,H,K,D,rot,prompts,steps", [
    (16, 8, 2, 128, 128, [37, 5, 0, 130], 20),
    (64, 16, 2, 256, 64, [200, 64], 6),
    (32, 4, 4, 64, 32, [1, 31, 33], 35),
])
def test_decode_loop(P, H, K, D, rot, prompts, steps):
    """Two layers: the prompts' chunk, then decode steps captured once as a graph and replayed
    while the cache grows, with rows that finish, restart and take back drafts."""
    B, layers = len(prompts), 2
    g = torch.Generator(device=DEV).manual_seed(P + D)
    width = -(-(max(prompts) + 2 * steps + 8) // P)
    kv = m.DeviceKv(B, width, B * width, P, K, D, layers=layers)
    rope = m.make_rope(m.rope_table(width * P, rot), rot)
    wq, wk = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    scale = D ** -0.5
    hist = [[[] for _ in range(B)] for _ in range(layers)]  # slots are read back each step

    def layer_calls(l, batch, T, max_new, buf, q, out, ws):
        c = kv.layers[l]
        x = buf[l]
        proj = m.make_qkv(x[:, :H], x[:, H:H + K], x[:, H + K:], wq, wk)
        m.moe_qkv_store(c, batch.c, rope, proj, T, None, q[l])
        m.moe_kv_attention(c, batch.c, B, q[l], T, H, max_new, scale, ws, ws.numel(), out[l])

    def check(batch, T, q, out):
        assert int(batch.err[0]) == 0
        start, length, table = _np(batch.q_start), _np(batch.kv_len), _np(kv.block_table)
        for l in range(layers):
            pool = _np(kv.pools[l])
            for b in range(B):
                n, L = start[b + 1] - start[b], int(length[b])
                if n == 0:
                    continue
                j = np.arange(L)
                k, v = ref.read_slots(pool, table[b, j // P] * P + j % P, K, P, D)
                qq = _f64(q[l][start[b]:start[b + 1]])
                want = ref.attention(qq, k, v, scale, L - n)
                off = np.abs(_f64(out[l][start[b]:start[b + 1]]) - want)
                assert np.all(off <= ref.attention_bound(qq, k, v, scale, want)), (l, b, L)
                # the last token's key is this step's own
                x = _f64(buf_now[l][start[b + 1] - 1:start[b + 1], H:H + K])
                y = ref.norm_rotate(x, _np(wk), 1e-6, _np(rope.table_tensor), np.array([[L - 1]]),
                                    rot, False, None)
                _check_quantised(k[-1:], y, "k in the loop")

    def buffers(T):
        buf = torch.randn(layers, T, H + 2 * K, D, generator=g, device=DEV).bfloat16()
        q = torch.zeros(layers, T, H, D, dtype=torch.bfloat16, device=DEV)
        return buf, q, torch.zeros_like(q)

    T = sum(prompts)
    batch = m.DeviceKvBatch(T, B)
    buf_now, q, out = buffers(T)
    ws = torch.empty(m.moe_kv_attention_workspace_bytes(kv.c, B, T, H, max(prompts)),
                     dtype=torch.uint8, device=DEV)
    m.moe_kv_plan(kv.c, _ints(prompts), B, batch.c)
    for l in range(layers):
        layer_calls(l, batch, T, max(prompts), buf_now, q, out, ws)
    check(batch, T, q, out)

    # decode: at most 2 tokens a row (a draft), everything captured once
    T = 2 * B
    batch = m.DeviceKvBatch(T, B)
    buf_now, q, out = buffers(T)
    new = _ints([1] * B)
    ws = torch.empty(m.moe_kv_attention_workspace_bytes(kv.c, B, T, H, 2), dtype=torch.uint8,
                     device=DEV)
    tab = ref.Tables(B, width, B * width, P)
    tab.plan(prompts, sum(prompts))

    def step():
        m.moe_kv_plan(kv.c, new, B, batch.c)
        for l in range(layers):
            layer_calls(l, batch, T, 2, buf_now, q, out, ws)

    state = [t.clone() for t in (kv.block_table, kv.seq_len, kv.free_list, kv.free_count)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((kv.block_table, kv.seq_len, kv.free_list, kv.free_count), state):
        t.copy_(s)
    rng = np.random.default_rng(steps)
    for i in range(steps):
        n = rng.choice([1, 1, 1, 2, 0], B)
        if i == steps // 2:
            n[0] = -(1 << 30)  # this row finishes
        elif i % 5 == 4:
            n[B - 1] = -1  # a rejected draft
        new.copy_(_ints(n))
        buf_now.copy_(torch.randn(buf_now.shape, generator=g, device=DEV))
        graph.replay()
        tab.plan(n, T)
        assert np.array_equal(_np(kv.seq_len), tab.len)
        assert np.array_equal(_np(kv.block_table), tab.table)
        if i % 4 == 0 or i == steps - 1:
            check(batch, T, q, out)
