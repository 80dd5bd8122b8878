"""Arrays of queries, outputs and projections past 2^31 elements, the largest batches, and groups of many heads."""
import pytest
import torch

from test_gpu_cache_attn import Problem
from test_gpu_positions import split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def test_a_projection_past_32_bits(tp):
    """The last rows of 2.5 G elements give what they give alone, forward, backward and appended."""
    T, heads, kv, d, dt, last = 200000, 32, 32, 128, torch.bfloat16, 70
    g = torch.Generator(device="cuda").manual_seed(1)
    QKV = torch.randn(T, (heads + 2 * kv) * d, generator=g, device="cuda", dtype=dt)
    grads = [torch.randn(T, heads, d, generator=g, device="cuda", dtype=dt) for _ in "qk"]
    gains = [1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in "qk"]
    gains = [x.to(dt) for x in gains]
    pos = torch.arange(T, device="cuda")
    rope = tp.RopeTable(d)
    ctx, few = tp.QkContext(T, heads, kv, d, dt, rope), tp.QkContext(last, heads, kv, d, dt, rope)
    out, small = tp.qk_forward(ctx, QKV, pos, *gains), tp.qk_forward(few, QKV[-last:], pos[-last:], *gains)
    for a, b in zip(out, small):
        assert torch.equal(a[-last:], b)
    back, small_back = tp.qk_backward(ctx, *grads), tp.qk_backward(few, *(x[-last:] for x in grads))
    assert torch.equal(back["dQ"][-last:], small_back["dQ"]) and torch.equal(back["dK"][-last:], small_back["dK"])
    cache = tp.KvCache((T + 63) // 64, 64, kv, d, dt)
    Q = tp.kv_append(ctx, cache, QKV, pos, pos, *gains)
    at = pos[-last:]
    assert torch.equal(Q[-last:], small[0]) and torch.equal(cache.K[at // 64, :, at % 64], small[1])
    assert torch.equal(cache.V[at // 64, :, at % 64], split(QKV[-last:], heads, kv, d, 1)[2])
    assert tp.check_device_status(ctx) == tp.OK


@pytest.mark.parametrize("new", [1, 9])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_queries_past_32_bits(tp, dt, new):
    """Sequences on the same few pages: the first ones and the last ones give the same as in a batch of their own."""
    heads, kv, d = 32, 8, 128
    batch = (1 << 31) // (heads * d * new) + 100
    p = Problem([(20, new), (3, new), (40, new)], heads, kv, d, 8, dt, seed=40)
    want = p.run(tp)
    p.check(want)
    times = (batch + 2) // 3
    Q = torch.zeros(3 * times * new, heads, d, dtype=dt, device="cuda")
    Q[:3 * new], Q[-3 * new:] = p.Q, p.Q
    ctx = tp.CacheAttnContext(Q.shape[0], 3 * times, heads, kv, d, dt)
    O = torch.full_like(Q, 5.0)
    tp.cache_attention(ctx, tp.KvCache.of(p.K, p.V), Q, (torch.arange(3 * times + 1, device="cuda") * new).int(),
                       p.kv_len.repeat(times), p.table.repeat(times, 1), O=O)
    assert tp.check_device_status(ctx) == tp.OK and Q.numel() > 1 << 31
    for part in (O[:3 * new], O[-3 * new:]):
        p.check(part)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_the_largest_batch(tp, dt):
    """2^20 sequences, most of them without tokens."""
    batch, heads, kv, d = 1 << 20, 4, 2, 64
    p = Problem([(70, 2), (5, 1), (200, 3)], heads, kv, d, 16, dt, seed=41)
    where = [0, batch // 2 + 3, batch - 1]
    lens = torch.zeros(batch, dtype=torch.int32)
    new = torch.zeros(batch, dtype=torch.int64)
    table = torch.full((batch, p.table.shape[1]), -1, dtype=torch.int32, device="cuda")
    for i, b in enumerate(where):
        lens[b], new[b], table[b] = int(p.kv_len[i]), p.lens[i][1], p.table[i]
    q_start = torch.cat((torch.zeros(1, dtype=torch.int64), new.cumsum(0))).int().cuda()
    ctx = tp.CacheAttnContext(p.T, batch, heads, kv, d, dt)
    O = tp.cache_attention(ctx, tp.KvCache.of(p.K, p.V), p.Q, q_start, lens.cuda(), table)
    assert tp.check_device_status(ctx) == tp.OK
    p.check(O)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,kv", [([(300, 1), (40, 2)], 300, 1), ([(100, 3)], 1000, 2), ([(10, 1)], 4097, 1), ([(130, 33)], 129, 1)])
@pytest.mark.parametrize("tree", [False, True])
def test_groups_of_many_heads(tp, lens, heads, kv, kind, tree):
    p = Problem(lens, heads, kv, 64, 16, torch.float32 if kind == "f32" else torch.bfloat16, tree, seed=42)
    p.check(p.run(tp))
    assert tp.check_device_status(p.ctx) == tp.OK
