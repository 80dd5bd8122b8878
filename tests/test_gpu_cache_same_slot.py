"""Tokens appended to the same slot, which the caller is told not to do: every element of the slot's rows is one of theirs, and
nothing else changes."""
import pytest
import torch

from test_gpu_positions import cache_of, make, split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,heads,kv,d", [(2, 4, 2, 64), (600, 8, 8, 128), (33, 2, 1, 26)])
def test_the_same_slot_again_and_again(tp, T, heads, kv, d, dt):
    QKV, gq, gk, pos, _, _ = make(T, heads, kv, d, dt, 23)
    cache = cache_of(tp, 5, kv, 16, d, dt, "heads")
    K0, V0 = cache.K.clone(), cache.V.clone()
    slot = torch.full((T,), 37, device="cuda")  # row 5 of page 2
    ctx = tp.QkContext(T, heads, kv, d, dt, tp.RopeTable(d))
    Q = tp.kv_append(ctx, cache, QKV, pos, slot, gq, gk)
    assert tp.check_device_status(ctx) == tp.OK
    Qr, Kr = tp.qk_forward(ctx, QKV, pos, gq, gk)
    assert torch.equal(Q, Qr)
    for row, tokens in ((cache.K[2, :, 5], Kr), (cache.V[2, :, 5], split(QKV, heads, kv, d, 1)[2])):
        assert bool((row == tokens).any(0).all())
    for now, before in ((cache.K, K0), (cache.V, V0)):
        now[2, :, 5] = before[2, :, 5]
        assert torch.equal(now, before)
