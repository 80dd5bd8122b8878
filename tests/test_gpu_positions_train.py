"""Norms and rotation as a training step uses them: a projection, its queries and keys normed and rotated, causal attention,
and all gradients back to the projection's weight and the gains, against autograd in 64 bits; and the same tokens
appended and attended to from a cache, against the training pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def formula(x, gain, pos, theta, eps):
    """x [T, heads, d] normed, its halves turned as pairs."""
    y = gain * x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    f = pos[:, None, None] * theta
    u, v = y.chunk(2, -1)
    return torch.cat((u * f.cos() - v * f.sin(), u * f.sin() + v * f.cos()), -1)


def attention(Q, K, V, d):
    G = Q.shape[1] // K.shape[1]
    K, V = K.repeat_interleave(G, 1), V.repeat_interleave(G, 1)
    S = torch.einsum("ihd,jhd->hij", Q, K) * d ** -0.5
    S = S.masked_fill(torch.ones(S.shape[1:], dtype=torch.bool, device=S.device).triu(1), -float("inf"))
    return torch.einsum("hij,jhd->ihd", S.softmax(-1), V)


@pytest.mark.parametrize("heads,kv,d,t", [(4, 4, 64, 1), (8, 2, 128, 2), (6, 2, 80, 2)])
def test_training_step(tp, heads, kv, d, t):
    T, h, eps = 77, 96, 1e-6
    g = torch.Generator(device="cpu").manual_seed(d)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()
    X, W = rand(T, h), rand(h, (heads + 2 * kv) * d) * h ** -0.5
    gains = [1 + 0.1 * rand(d) for _ in "qk"]
    dO, pos = rand(T, heads, d), torch.arange(T, device="cuda") + 1000
    n, m = heads // t, kv // t
    cols = torch.arange((heads + 2 * kv) * d, device="cuda").reshape(t, n + 2 * m, d)
    of_q, of_k, of_v = (cols[:, a:b].reshape(-1) for a, b in ((0, n), (n, n + m), (n + m, n + 2 * m)))

    rope = tp.RopeTable(d)
    ctx = tp.QkContext(T, heads, kv, d, torch.float32, rope, eps=eps, t=t)
    QKV = X @ W
    Qr, Kr = (x.requires_grad_() for x in tp.qk_forward(ctx, QKV, pos, *gains))
    V = QKV[:, of_v].reshape(T, kv, d).requires_grad_()
    attention(Qr.double(), Kr.double(), V.double(), d).backward(dO.double())
    dQKV = torch.empty_like(QKV)
    grads = tp.qk_backward(ctx, Qr.grad, Kr.grad, out=dQKV)
    dQKV[:, of_v] = V.grad.reshape(T, kv * d)
    dW, dX = X.double().t() @ dQKV.double(), dQKV.double() @ W.double().t()

    theta = 10000.0 ** (-2 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    X64, W64, gq, gk = (x.double().requires_grad_() for x in (X, W, *gains))
    P = X64 @ W64
    part = lambda of, n: P[:, of].reshape(T, n, d)
    O = attention(formula(part(of_q, heads), gq, pos, theta, eps), formula(part(of_k, kv), gk, pos, theta, eps), part(of_v, kv), d)
    O.backward(dO.double())
    # 96 products and 64 steps of 2^-24 behind a score at most, which scores below 20 multiply by 40
    for name, got, want in (("X", dX, X64.grad), ("W", dW, W64.grad), ("gain_q", grads["dgain_q"], gq.grad), ("gain_k", grads["dgain_k"], gk.grad)):
        assert float((got - want).norm() / want.norm()) < 160 * 2.0 ** -24 * 40, name

    # the same tokens in two calls, from a cache
    cache = tp.KvCache(10, 8, kv, d, torch.float32)
    table = torch.randperm(10, generator=g).int().cuda()[None]
    row = torch.arange(T, device="cuda")
    slot = table[0].long()[row // 8] * 8 + row % 8
    out = []
    for a, b in ((0, 50), (50, T)):
        c = tp.QkContext(b - a, heads, kv, d, torch.float32, rope, eps=eps, t=t)
        Q = tp.kv_append(c, cache, QKV[a:b], pos[a:b], slot[a:b], *gains)
        assert torch.equal(Q, Qr[a:b])
        attn = tp.CacheAttnContext(b - a, 1, heads, kv, d, torch.float32)
        i32 = dict(dtype=torch.int32, device="cuda")
        out.append(tp.cache_attention(attn, cache, Q, torch.tensor([0, b - a], **i32), torch.tensor([b], **i32), table))
        assert tp.check_device_status(c) == tp.OK and tp.check_device_status(attn) == tp.OK
    at = table[0].long()[row // 8]
    assert torch.equal(cache.K[at, :, row % 8], Kr) and torch.equal(cache.V[at, :, row % 8], V)
    assert float((torch.cat(out) - O).norm() / O.norm()) < 160 * 2.0 ** -24 * 40
