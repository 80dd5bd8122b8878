"""Norms and rotation at both ends of the range, and the accuracy of the angles, on the GPU against 64 bits."""
import pytest
import torch

from test_gpu_positions import E, make, rotate, split, theta

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


@pytest.mark.parametrize("size,grad", [(3e-20, 1.0), (1e18, 1e-4), (1e-10, 1e-10), (1e10, 1e10)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradients_of_small_and_large_rows(tp, size, grad, layout):
    """Without eps the gradient of the norm goes with 1/|x|: no power of it may leave fp32's range on the way.  A mean square
    of 9e-40 has 19 bits: the root of it is off by 2^-21 more, 8 of the steps that test_gpu_positions counts."""
    T, heads, kv, d = 9, 3, 2, 64
    QKV, gq, gk, pos, dQ, dK = make(T, heads, kv, d, torch.float32, 17)
    QKV, dQ, dK = QKV * size, dQ * grad, dK * grad
    ctx = tp.QkContext(T, heads, kv, d, torch.float32, tp.RopeTable(d, layout=layout), eps=0.0)
    tp.qk_forward(ctx, QKV, pos, gq, gk)
    g = tp.qk_backward(ctx, dQ, dK)
    for x, gain, dy, dx, dg in zip(split(QKV, heads, kv, d, 1), (gq, gk), (dQ, dK), (g["dQ"], g["dK"]), (g["dgain_q"], g["dgain_k"])):
        x, gain, dy = x.double(), gain.double(), dy.double()
        back, step = rotate(dy, pos, theta(d), d, layout, back=True)
        r = x.square().mean(-1, keepdim=True).rsqrt()
        h = x * r
        ref = r * (back * gain - h * (back * gain * h).mean(-1, keepdim=True))
        off = r * (step * gain.abs() + h.abs() * (step * (gain * h).abs()).mean(-1, keepdim=True))
        assert bool(((dx.double() - ref).abs() <= E * ref.abs() + 72 * E * off).all())
        ref, off = (back * h).sum((0, 1)), (step * h.abs()).sum((0, 1))
        assert bool(((dg.double() - ref).abs() <= E * ref.abs() + (72 + T * heads / 8) * E * off).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_sines_and_cosines(tp, layout):
    """A pair (1, 0) becomes (cos, sin), with no other rounding than theirs: one step of 2^-24 of the function itself, and of its
    argument's, which is at most an eighth of a turn and rounded to 24 bits: 2^-25 pi / 4."""
    T, d = 4096, 128
    g = torch.Generator(device="cpu").manual_seed(7)
    pos = torch.cat((torch.arange(2048), torch.randint(0, 1 << 24, (T - 2048,), generator=g))).cuda()
    Q, K = torch.zeros(T, 1, d, device="cuda"), torch.zeros(T, 1, d, device="cuda")
    first = slice(0, d // 2) if layout == "half" else slice(0, d, 2)
    second = slice(d // 2, d) if layout == "half" else slice(1, d, 2)
    Q[..., first] = 1.0
    K[..., second] = 1.0
    ctx = tp.QkContext(T, 1, 1, d, torch.float32, tp.RopeTable(d, layout=layout), norm=False)
    Qr, Kr = tp.qk_forward(ctx, (Q, K), pos)
    a = pos.double()[:, None, None] * torch.tensor(theta(d), dtype=torch.float64, device="cuda")
    # the angle itself in 64 bits: 2^24 times 2^-53, twice
    tol = 2.0 ** -24 + 2.0 ** -25 * 0.7854 + 2.0 ** -28
    for got, ref in ((Qr[..., first], a.cos()), (Qr[..., second], a.sin()), (Kr[..., first], -a.sin()), (Kr[..., second], a.cos())):
        assert bool(((got.double() - ref).abs() <= tol).all()), float((got.double() - ref).abs().max() * 2 ** 24)
