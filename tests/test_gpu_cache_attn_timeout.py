"""Waits of the tensor-core attention kernels that run out.

With a limit of a nanosecond a wait gives up when what it waits for has not come after some tries of the hardware's own length.
Where a block has several long units the planning warp waits for whole units, which is long enough; elsewhere it depends on the
machine, so that either status is right there: an OK with the right result and a TIMEOUT with any.  Whatever came first, the call
ends, what it had under way ends with it, and the same context serves the next call, whose limit is the usual one, with
the same bits as before."""
import pytest
import torch

from test_gpu_cache_attn import Problem

pytestmark = pytest.mark.gpu

DEFAULT_NS = 2_000_000_000


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    yield tpmlp
    tpmlp.set_wait_limit_ns(DEFAULT_NS)


def short_and_usual(tp, run, ctx, times):
    """Statuses of calls with a limit of a nanosecond; calls with the usual one between them."""
    want = run()
    assert tp.check_device_status(ctx) == tp.OK
    seen = []
    for _ in range(times):
        tp.set_wait_limit_ns(1)
        try:
            got = run()
        finally:
            tp.set_wait_limit_ns(DEFAULT_NS)
        seen.append(tp.check_device_status(ctx))
        assert seen[-1] in (tp.OK, tp.ERR_TIMEOUT)
        assert seen[-1] == tp.ERR_TIMEOUT or torch.equal(got, want)
        assert torch.equal(run(), want) and tp.check_device_status(ctx) == tp.OK
    print("statuses:", seen)
    return seen


@pytest.mark.parametrize("lens,heads,kv,d", [([(2047, 1)], 1, 1, 128), ([(300, 1), (40, 2)], 8, 2, 64), ([(2000, 1)] * 40, 8, 8, 128),
                                             ([(700, 3)] * 9, 4, 2, 256), ([(2000, 100)], 8, 1, 128), ([(500, 60)] * 12, 8, 2, 64),
                                             ([(500, 60)] * 5, 8, 2, 256)])
def test_few_units(tp, lens, heads, kv, d):
    p = Problem(lens, heads, kv, d, 16, torch.bfloat16, seed=31)
    ctx = tp.CacheAttnContext(p.T, len(lens), heads, kv, d, torch.bfloat16)
    short_and_usual(tp, lambda: p.run(tp, ctx=ctx), ctx, 5)


@pytest.mark.parametrize("new,heads,d,batch", [(1, 1, 64, 800), (2, 4, 128, 800), (3, 2, 256, 500), (40, 2, 64, 400), (40, 2, 128, 400),
                                               (50, 4, 256, 300)])
def test_long_units(tp, new, heads, d, batch):
    """Sequences of 2048 tiles (of the same few pages again and again), several to a block: milliseconds for a unit, which its
    planning warp waits for while copies and products go on."""
    keys, page, pages = 1 << 18, 128, 48
    g = torch.Generator(device="cuda").manual_seed(32)
    K, V = (torch.randn(pages, 1, page, d, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    Q = torch.randn(batch * new, heads, d, generator=g, device="cuda").to(torch.bfloat16)
    table = (torch.arange(keys // page, device="cuda") % pages).int().repeat(batch, 1)
    q_start = (torch.arange(batch + 1, device="cuda") * new).int()
    kv_len = torch.full((batch,), keys, dtype=torch.int32, device="cuda")
    ctx = tp.CacheAttnContext(batch * new, batch, heads, 1, d, torch.bfloat16)
    cache = tp.KvCache.of(K, V)
    seen = short_and_usual(tp, lambda: tp.cache_attention(ctx, cache, Q, q_start, kv_len, table), ctx, 4)
    assert tp.ERR_TIMEOUT in seen
