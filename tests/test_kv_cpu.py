"""Host-side checks of the 4-bit key/value cache's entry points: sizes and refusals (every
argument is checked before any CUDA call, so they need no GPU)."""
import pytest

import moe_expert_offload_gb300 as m


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_expert_offload_gb300 import _build

    _build.build()


PTR = 1 << 20  # a non-NULL, aligned address that no refused call follows


def _kv(**kw):
    f = dict(num_blocks=8, block_tokens=64, kv_heads=2, head_dim=128, max_rows=4, max_blocks=8,
             block_table=PTR, seq_len=PTR, free_list=PTR, free_count=PTR, pool=PTR)
    f.update(kw)
    return m.MoeKv(**f)


def _batch(**kw):
    f = dict(max_tokens=16, max_rows=4, q_start=PTR, kv_len=PTR, slot=PTR, pos=PTR, err=PTR)
    f.update(kw)
    return m.MoeKvBatch(**f)


def _rope(axis=0, **kw):
    f = dict(table=PTR, max_pos=100, rotary_dim=64, adjacent=0, axes=1)
    f.update(kw)
    r = m.MoeRope(**f)
    r.pair_axis[3] = axis
    return r


def _proj(**kw):
    f = dict(q=PTR, k=PTR, v=PTR, q_token_stride=1024, q_head_stride=128, k_token_stride=256,
             k_head_stride=128, v_token_stride=256, v_head_stride=128, q_heads=8, eps=1e-6,
             q_norm=PTR, k_norm=None)
    f.update(kw)
    return m.MoeQkv(**f)


def _refused(code, call, *words):
    with pytest.raises(m.MoeError) as e:
        call()
    assert e.value.code == code, e.value
    for w in words:
        assert w in str(e.value)


def test_block_bytes():
    assert m.moe_kv_block_bytes(_kv()) == 2 * 4 * 18 * 128
    for D in (64, 128, 256):
        for P in (16, 32, 64, 128):
            assert m.moe_kv_block_bytes(_kv(head_dim=D, block_tokens=P, kv_heads=3)) == (
                3 * P * D * 9 // 8)


SHAPES = [
    (dict(num_blocks=0), m.MOE_EINVAL), (dict(block_tokens=48), m.MOE_EINVAL),
    (dict(block_tokens=0), m.MOE_EINVAL), (dict(kv_heads=0), m.MOE_EINVAL),
    (dict(kv_heads=257), m.MOE_EINVAL), (dict(head_dim=96), m.MOE_EUNSUPPORTED),
    (dict(head_dim=512), m.MOE_EUNSUPPORTED),
    (dict(num_blocks=1 << 25, block_tokens=128), m.MOE_EUNSUPPORTED),
]
TABLES = [
    (dict(max_rows=0), m.MOE_EINVAL), (dict(max_blocks=0), m.MOE_EINVAL),
    (dict(max_blocks=1 << 25, block_tokens=64), m.MOE_EUNSUPPORTED),
    (dict(block_table=None), m.MOE_EINVAL), (dict(seq_len=None), m.MOE_EINVAL),
    (dict(free_list=None), m.MOE_EINVAL), (dict(free_count=None), m.MOE_EINVAL),
]
POOL = [(dict(pool=None), m.MOE_EINVAL), (dict(pool=PTR + 64), m.MOE_EINVAL)]
BATCH = [
    (dict(max_tokens=0), m.MOE_EINVAL), (dict(max_rows=0), m.MOE_EINVAL),
    (dict(q_start=None), m.MOE_EINVAL), (dict(kv_len=None), m.MOE_EINVAL),
    (dict(slot=None), m.MOE_EINVAL), (dict(pos=None), m.MOE_EINVAL), (dict(err=None), m.MOE_EINVAL),
]


def _attend(kv=None, batch=None, rows=4, q=PTR, T=16, heads=8, max_new=4, scale=0.1, ws=PTR,
            n=1 << 40, out=PTR):
    return m.moe_kv_attention(kv or _kv(), batch or _batch(), rows, q, T, heads, max_new, scale, ws,
                              n, out, 0)


def _store(kv=None, batch=None, rope=None, proj=None, T=16, positions=None, q_out=PTR):
    return m.moe_qkv_store(kv or _kv(), batch or _batch(), rope or _rope(), proj or _proj(), T,
                           positions, q_out, 0)


@pytest.mark.parametrize("kw,code", SHAPES)
def test_shape_refusals(kw, code):
    kv = _kv(**kw)
    assert m.moe_kv_block_bytes(kv) == 0
    for call in (lambda: m.moe_kv_reset(kv, 0), lambda: m.moe_kv_plan(kv, PTR, 4, _batch(), 0),
                 lambda: _store(kv), lambda: m.moe_kv_load(kv, PTR, 4, PTR, PTR, None, 0),
                 lambda: _attend(kv)):
        _refused(code, call)
    assert m.moe_kv_attention_workspace_bytes(kv, 4, 16, 8, 4) == 0


@pytest.mark.parametrize("kw,code", TABLES)
def test_table_refusals(kw, code):
    kv = _kv(**kw)
    for call in (lambda: m.moe_kv_reset(kv, 0), lambda: m.moe_kv_plan(kv, PTR, 4, _batch(), 0),
                 lambda: _attend(kv)):
        _refused(code, call)


@pytest.mark.parametrize("kw,code", POOL)
def test_pool_refusals(kw, code):
    kv = _kv(**kw)
    for call in (lambda: _store(kv), lambda: m.moe_kv_load(kv, PTR, 4, PTR, PTR, None, 0),
                 lambda: _attend(kv)):
        _refused(code, call, "pool")


@pytest.mark.parametrize("kw,code", BATCH)
def test_batch_refusals(kw, code):
    b = _batch(**kw)
    for call in (lambda: m.moe_kv_plan(_kv(), PTR, 1, b, 0), lambda: _store(batch=b, T=1),
                 lambda: _attend(batch=b, rows=1, T=1)):
        _refused(code, call)


def test_rows_and_tokens():
    for rows, code in ((0, m.MOE_EINVAL), (-1, m.MOE_EINVAL), (5, m.MOE_ECAPACITY)):
        _refused(code, lambda: m.moe_kv_plan(_kv(), PTR, rows, _batch(max_rows=9), 0), "rows")
        _refused(code, lambda: _attend(rows=rows), "rows")
    for T, code in ((-1, m.MOE_EINVAL), (17, m.MOE_ECAPACITY)):
        _refused(code, lambda: _store(T=T), "T")
        _refused(code, lambda: _attend(T=T), "T")
    _refused(m.MOE_EINVAL, lambda: m.moe_kv_load(_kv(), PTR, -1, PTR, PTR, None, 0), "T")
    _refused(m.MOE_EINVAL, lambda: m.moe_kv_plan(_kv(), None, 4, _batch(), 0), "new_len")
    # nothing to do launches nothing
    assert _store(T=0) == m.MOE_OK and _attend(T=0) == m.MOE_OK
    assert m.moe_kv_load(_kv(), PTR, 0, PTR, PTR, None, 0) == m.MOE_OK


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(q=PTR + 8), dict(k=PTR + 2), dict(v=PTR + 4),
    dict(q_token_stride=1025), dict(k_head_stride=4), dict(v_token_stride=-8), dict(q_heads=0),
    dict(q_heads=257), dict(eps=-1.0), dict(eps=float("nan")), dict(q_norm=PTR + 4),
    dict(k_norm=PTR + 8),
])
def test_projection_refusals(kw):
    _refused(m.MOE_EINVAL, lambda: _store(proj=_proj(**kw)))


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=24), dict(rotary_dim=-16), dict(rotary_dim=144), dict(table=None),
    dict(table=PTR + 4), dict(max_pos=0), dict(adjacent=2), dict(axes=0), dict(axes=5),
    dict(axes=3), dict(axis=1),
])
def test_rope_refusals(kw):
    _refused(m.MOE_EINVAL, lambda: _store(rope=_rope(**kw)))


def test_store_and_load_pointers():
    _refused(m.MOE_EINVAL, lambda: _store(q_out=None), "q_out")
    _refused(m.MOE_EINVAL, lambda: _store(q_out=PTR + 8), "q_out")
    for a in ((None, PTR, PTR), (PTR, None, PTR), (PTR, PTR, None), (PTR, PTR + 8, PTR),
              (PTR, PTR, PTR + 8)):
        _refused(m.MOE_EINVAL, lambda: m.moe_kv_load(_kv(), a[0], 4, a[1], a[2], None, 0))


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), m.MOE_EINVAL), (dict(heads=7), m.MOE_EINVAL), (dict(heads=258), m.MOE_EINVAL),
    (dict(heads=130), m.MOE_EUNSUPPORTED), (dict(max_new=0), m.MOE_EINVAL),
    (dict(q=None), m.MOE_EINVAL), (dict(out=None), m.MOE_EINVAL), (dict(ws=None), m.MOE_EINVAL),
    (dict(q=PTR + 8), m.MOE_EINVAL), (dict(out=PTR + 2), m.MOE_EINVAL),
    (dict(ws=PTR + 128), m.MOE_EINVAL), (dict(scale=0.0), m.MOE_EINVAL),
    (dict(scale=-1.0), m.MOE_EINVAL), (dict(scale=float("inf")), m.MOE_EINVAL),
    (dict(scale=float("nan")), m.MOE_EINVAL), (dict(n=0), m.MOE_ECAPACITY),
])
def test_attention_refusals(kw, code):
    _refused(code, lambda: _attend(**kw))


def test_workspace_size():
    n = m.moe_kv_attention_workspace_bytes(_kv(), 4, 16, 8, 4)
    assert n > 0
    _refused(m.MOE_ECAPACITY, lambda: _attend(n=n - 1), "workspace")
    for a in ((0, 16, 8, 4), (4, -1, 8, 4), (4, 16, 9, 4), (4, 16, 8, 0)):
        assert m.moe_kv_attention_workspace_bytes(_kv(), *a) == 0


def test_no_tokens_need_no_buffers():
    """An empty step's tensors have no address."""
    proj = _proj(q=None, k=None, v=None)
    assert _store(T=0, proj=proj, q_out=None) == m.MOE_OK
    assert m.moe_kv_load(_kv(), None, 0, None, None, None, 0) == m.MOE_OK
    assert _attend(T=0, q=None, out=None) == m.MOE_OK


def test_binding_refusals():
    import torch

    t = m.rope_table(7, 32, device="cpu")
    for a in ((t.double(), 32), (t[:, :16], 16), (t, 48), (t, 32, False, 2, [0, 2]),
              (t, 32, False, 1, [0, 256]), (t, 32, False, 1, [-1]), (t, 32, False, 1, [0] * 129)):
        with pytest.raises(m.MoeError):
            m.make_rope(*a)
    x = torch.zeros(5, 12, 64, dtype=torch.bfloat16)
    q, k, v, w = x[:, :8], x[:, 8:10], x[:, 10:], torch.ones(64)
    m.make_qkv(q, k, v, w, w)
    m.make_qkv(q.view(torch.int16), k, v)
    for a in ((q.half(), k, v), (q, k.float(), v), (q, k, x[:, 9:]), (q, k[:4], v[:4]),
              (q, k[..., :32], v[..., :32]), (q, k, v, w.half()), (q, k, v, w[:32]),
              (q, k, v, None, torch.ones(128)[::2])):
        with pytest.raises(m.MoeError):
            m.make_qkv(*a)


def test_binding_checks_arrays():
    """Arrays of another type, too short or not contiguous are refused before the library sees
    them; so is a projection that is not the cache's."""
    import torch

    def refused(*words):
        return lambda call: _refused(m.MOE_EINVAL, call, *words)

    kv, b, T = _kv(), _batch(), 5
    for t in (torch.ones(4, dtype=torch.int64), torch.ones(3, dtype=torch.int32),
              torch.ones(8, dtype=torch.int32)[::2], torch.ones(4)):
        refused("new_len")(lambda: m.moe_kv_plan(kv, t, 4, b, 0))
        refused("slots")(lambda: m.moe_kv_load(kv, t, 4, PTR, PTR, None, 0))
    x = torch.zeros(T, 12, 128, dtype=torch.bfloat16)
    q, out = x[:, :8].contiguous(), torch.zeros(T, 8, 128, dtype=torch.bfloat16)
    proj = m.make_qkv(x[:, :8], x[:, 8:10], x[:, 10:])
    for t in (x[:, :8], q[:4], q.half(), q.transpose(0, 1)):
        refused("q")(lambda: _attend(q=t, T=T))
        refused("out")(lambda: _attend(out=t, T=T))
        refused("q_out")(lambda: _store(proj=proj, T=T, q_out=t))
    for t in (q[:, :1], q[:4, :2].contiguous(), q[:, :2].float()):
        refused("k")(lambda: m.moe_kv_load(kv, PTR, T, t, PTR, None, 0))
        refused("v")(lambda: m.moe_kv_load(kv, PTR, T, PTR, t, None, 0))
    for args in (dict(T=6), dict(T=T, kv=_kv(kv_heads=4)), dict(T=T, kv=_kv(kv_heads=1)),
                 dict(T=T, kv=_kv(head_dim=64)), dict(T=T, kv=_kv(head_dim=256))):
        refused("proj")(lambda: _store(proj=proj, **args))
    rope = _rope(axes=3)
    for t in (torch.zeros(3, T, dtype=torch.int64), torch.zeros(2, T, dtype=torch.int32),
              torch.zeros(3, T + 1, dtype=torch.int32), torch.zeros(T, 3, dtype=torch.int32).t()):
        refused("positions")(lambda: _store(proj=proj, T=T, rope=rope, positions=t, q_out=out))
    refused("positions")(lambda: _store(proj=proj, T=T, positions=torch.zeros(T), q_out=out))
    # what fits goes on to the library's own checks
    fits = torch.zeros(3, T, dtype=torch.int32)
    _refused(m.MOE_EINVAL, lambda: _store(proj=proj, T=T, rope=_rope(axes=3, max_pos=0),
                                          positions=fits, q_out=out), "max_pos")
    _refused(m.MOE_EINVAL, lambda: _store(proj=proj, T=T, rope=_rope(rotary_dim=0), positions=x,
                                          q_out=PTR + 8), "q_out")  # nothing turns: not looked at
    _refused(m.MOE_EINVAL, lambda: _attend(q=q, out=out.view(torch.int16), T=T, scale=0.0), "scale")


def test_binding_helpers():
    import torch

    t = m.rope_table(7, 32, base=100.0, device="cpu")
    assert t.shape == (7, 32) and t.dtype == torch.float32
    assert torch.equal(t[0], torch.cat((torch.ones(16), torch.zeros(16))))
    p = torch.tensor(6.0, dtype=torch.float64) * 100.0 ** (-2.0 * 5 / 32)
    assert t[6, 5] == p.cos().float() and t[6, 16 + 5] == p.sin().float()
    r = m.make_rope(t, 32, adjacent=True, axes=3, pair_axis=[i % 3 for i in range(16)])
    assert (r.max_pos, r.rotary_dim, r.adjacent, r.axes, r.pair_axis[4]) == (7, 32, 1, 3, 1)
    x = torch.zeros(5, 12, 64, dtype=torch.bfloat16)
    q = m.make_qkv(x[:, :8], x[:, 8:10], x[:, 10:])
    assert q.q_heads == 8 and q.k - q.q == 8 * 64 * 2 and q.v_token_stride == 12 * 64
    with pytest.raises(m.MoeError):
        m.make_qkv(x.transpose(1, 2), x, x)
    with pytest.raises(m.MoeError):
        m.DeviceKv(4, 4, 4, 64, 2, 96, device="cpu")
    kv = m.DeviceKv(2, 4, 6, 16, 1, 64, device="cpu", layers=3)
    assert kv.free_list.tolist() == [5, 4, 3, 2, 1, 0] and kv.layers[2].pool == kv.pools[2].data_ptr()
