"""The checks of test_gpu_positions on outputs that have to be finite (a comparison with NaN is false either way round): rows
that are read element by element, 8 or 16 bytes at a time, and far positions."""
import pytest
import torch

from test_gpu_positions import EPS, check_backward, check_forward, make, split, theta

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def finite(*tensors):
    assert all(bool(x.isfinite().all()) for x in tensors if x is not None)


def both_ways(tp, ctx, QKV, pos, gains, grads, heads, kv, d, f, rot, layout, amp=1.0):
    out = tp.qk_forward(ctx, QKV, pos, *gains)
    g = tp.qk_backward(ctx, *grads)
    finite(*out, *g.values())
    parts = split(QKV.contiguous(), heads, kv, d, 1)
    for i, name in enumerate("QK"):
        check_forward(out[i], parts[i], gains[i], pos, f, rot, layout, amp)
        check_backward(g["d" + name], g["dgain_" + name.lower()], parts[i], gains[i], grads[i], pos, f, rot, layout, amp)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,cut", [(64, 64, 1), (128, 116, 0), (128, 120, 0), (128, 128, 0), (250, 26, 0), (256, 256, 3)])
def test_rows_of_any_alignment(tp, d, rot, cut, layout, norm, dt):
    T, heads, kv = 37, 4, 2
    QKV, gq, gk, pos, dQ, dK = make(T, heads, kv, d, dt, d + rot, norm=norm)
    rows = torch.full((T, QKV.shape[1] + 2 * cut), float("nan"), dtype=dt, device="cuda")
    view = rows[:, cut:cut + QKV.shape[1]]
    view.copy_(QKV)
    ctx = tp.QkContext(T, heads, kv, d, dt, tp.RopeTable(rot, layout=layout), norm=norm, eps=EPS)
    both_ways(tp, ctx, view, pos, (gq, gk), (dQ, dK), heads, kv, d, theta(rot), rot, layout)


@pytest.mark.parametrize("scaling", [("linear", 4.0), ("parts", 8.0, 2048, 1.0, 32.0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_far_positions(tp, norm, layout, scaling):
    T, heads, kv, d = 56, 2, 1, 128
    QKV, gq, gk, _, dQ, dK = make(T, heads, kv, d, torch.float32, 5, norm=norm)
    pos = torch.tensor([0, 1, 3, -1, -5, 1 << 20, (1 << 24) + 1] * 8).cuda()
    ctx = tp.QkContext(T, heads, kv, d, torch.float32, tp.RopeTable(d, 500000.0, layout, scaling, 1.25), norm=norm, eps=EPS)
    both_ways(tp, ctx, QKV, pos, (gq, gk), (dQ, dK), heads, kv, d, theta(d, 500000.0, scaling), d, layout, 1.25)
