"""Attention over a paged cache with scores that are exact in fp32 and far apart.

Queries and keys are small whole numbers and the scale is a power of two, so that every score is exact whatever the order of its
sum, and scores that differ do so by 32 at least: a weight is that of one key alone (or of keys with the very same score)
and all others are below 2^-46.  What is left of the error is the weights' rounding (bf16: 2^-8 of each, and the same of
their sum), n + 64 steps of 2^-24 of the sum, and the output's own rounding."""
import pytest
import torch

from test_gpu_cache_attn import E, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


LENS = [([(700, 5), (1500, 1)], 8, 2), ([(700, 50), (1500, 20)], 8, 2), ([(0, 300)], 4, 4), ([(3000, 1)], 16, 1)]


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kind", ["bf16", "bf16-ffma", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,heads,kv", LENS)
def test_weights_of_one_key_alone(tp, lens, heads, kv, d, kind, sign):
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    p = Problem(lens, heads, kv, d, 16, dt, True, seed=d)
    g = torch.Generator(device="cpu").manual_seed(d)
    p.Q = torch.randint(-4, 5, p.Q.shape, generator=g).to(dt).cuda()
    p.K = torch.randint(-4, 5, p.K.shape, generator=g).to(dt).cuda()
    scale = 32.0 * sign
    O = p.run(tp, tp.ALGO_SIMT if kind == "bf16-ffma" else None, scale=scale)
    assert tp.check_device_status(p.ctx) == tp.OK
    q0, sharp, count = 0, 0, 0
    for b, (c, n) in enumerate(lens):
        key = torch.arange(c + n, device="cuda")
        page = p.table[b].long()[key // 16]
        K, V = (x[page, :, key % 16].double() for x in (p.K, p.V))
        seen = p.seen(b)
        for h in range(heads):
            k, v = K[:, h * kv // heads], V[:, h * kv // heads]
            S = (p.Q[q0:q0 + n, h].double() @ k.t() * scale).masked_fill(~seen, -float("inf"))
            P = torch.softmax(S, 1)
            ref, size = P @ v, P @ v.abs()
            u = torch.finfo(dt).eps / 2
            tol = u * ref.abs() + ((c + n + 64) * E + (2 * 2.0 ** -8 if dt == torch.bfloat16 else 0.0)) * 1.01 * size
            assert bool(((O[q0:q0 + n, h].double() - ref).abs() <= tol).all()), (b, h)
            sharp, count = sharp + int((2 * tol < ref.abs()).sum()), count + ref.numel()
        q0 += n
    # zeros, or values with the other sign, would be found
    assert sharp > 0.9 * count
