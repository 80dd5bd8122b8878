"""What qk_backward reads of the qk_forward before it: once something of the context's own has been written over it, a
further backward pass is refused instead of taking gradients for inputs."""
import pytest
import torch

from test_gpu_positions import make, split

pytestmark = pytest.mark.gpu

HEADS, KV, D, T = 4, 2, 64, 21


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def forward(tp, dt, t=1, norm=True):
    QKV, gq, gk, pos, dQ, dK = make(T, HEADS, KV, D, dt, 21, norm=norm)
    ctx = tp.QkContext(T, HEADS, KV, D, dt, tp.RopeTable(D), norm=norm, t=t)
    tp.qk_forward(ctx, QKV, pos, gq, gk)
    return ctx, QKV, pos, gq, gk, dQ, dK


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t", [1, 2])
def test_gradients_over_the_projection(tp, dt, t):
    ctx, QKV, pos, gq, gk, dQ, dK = forward(tp, dt, t)
    before = QKV.clone()
    want = tp.qk_backward(ctx, dQ, dK)
    again = tp.qk_backward(ctx, dQ, dK)  # nothing has been written over yet
    assert all(torch.equal(want[k], again[k]) for k in want)
    got = tp.qk_backward(ctx, dQ, dK, out=QKV)
    assert got["dQKV"] is QKV
    q, k, v = split(QKV, HEADS, KV, D, t)
    assert torch.equal(q, want["dQ"]) and torch.equal(k, want["dK"]) and torch.equal(v, split(before, HEADS, KV, D, t)[2])
    assert torch.equal(got["dgain_q"], want["dgain_q"]) and torch.equal(got["dgain_k"], want["dgain_k"])
    with pytest.raises(ValueError, match="gone"):
        tp.qk_backward(ctx, dQ, dK)
    # the next forward pass starts anew
    QKV.copy_(before)
    tp.qk_forward(ctx, QKV, pos, gq, gk)
    got = tp.qk_backward(ctx, dQ, dK)
    assert all(torch.equal(want[k], got[k]) for k in want)


@pytest.mark.parametrize("which", ["q", "k"])
def test_one_gradient_over_its_input(tp, which):
    ctx, QKV, pos, gq, gk, dQ, dK = forward(tp, torch.bfloat16)
    want = tp.qk_backward(ctx, dQ, dK)
    Q, K = QKV[:, :HEADS * D].view(T, HEADS, D), QKV[:, HEADS * D:(HEADS + KV) * D].view(T, KV, D)
    out = (Q, torch.empty_like(dK)) if which == "q" else (torch.empty_like(dQ), K)
    got = tp.qk_backward(ctx, dQ, dK, out=out)
    assert torch.equal(got["dQ"], want["dQ"]) and torch.equal(got["dK"], want["dK"])
    with pytest.raises(ValueError, match="gone"):
        tp.qk_backward(ctx, dQ, dK)


def test_without_the_norm_nothing_is_read(tp):
    ctx, QKV, pos, gq, gk, dQ, dK = forward(tp, torch.float32, norm=False)
    want = tp.qk_backward(ctx, dQ, dK)
    tp.qk_backward(ctx, dQ, dK, out=QKV)
    got = tp.qk_backward(ctx, dQ, dK)
    assert torch.equal(got["dQ"], want["dQ"]) and torch.equal(got["dK"], want["dK"])


def test_queries_of_an_append_over_the_saved_ones(tp):
    ctx, QKV, pos, gq, gk, dQ, dK = forward(tp, torch.bfloat16)
    cache = tp.KvCache(4, 16, KV, D, torch.bfloat16)
    slot = torch.arange(T, device="cuda")
    tp.kv_append(ctx, cache, QKV, pos, slot, gq, gk)
    tp.qk_backward(ctx, dQ, dK)
    tp.kv_append(ctx, cache, QKV, pos, slot, gq, gk, out=QKV[:, :HEADS * D].view(T, HEADS, D))
    with pytest.raises(ValueError, match="gone"):
        tp.qk_backward(ctx, dQ, dK)


def test_queries_of_another_append_over_the_saved_keys(tp):
    QKV, gq, gk, pos, dQ, dK = make(T, KV, KV, D, torch.bfloat16, 22)
    ctx = tp.QkContext(T, KV, KV, D, torch.bfloat16, tp.RopeTable(D))
    tp.qk_forward(ctx, QKV, pos, gq, gk)
    cache = tp.KvCache(4, 16, KV, D, torch.bfloat16)
    tp.kv_append(ctx, cache, QKV.clone(), pos, torch.arange(T, device="cuda"), gq, gk, out=QKV[:, KV * D:2 * KV * D].view(T, KV, D))
    with pytest.raises(ValueError, match="gone"):
        tp.qk_backward(ctx, dQ, dK)


def test_a_refused_forward_pass(tp):
    ctx, QKV, pos, gq, gk, dQ, dK = forward(tp, torch.bfloat16)
    with pytest.raises(ValueError):
        tp.qk_forward(ctx, QKV[:-1], pos, gq, gk)
    with pytest.raises(ValueError, match="qk_forward"):
        tp.qk_backward(ctx, dQ, dK)
