"""Norms and rotation at both ends of the range on the GPU against 64 bits."""
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
