"""Visible scores of minus infinity (an infinite component of a key, or a product past the type's range): they have no
weight, and a row that sees nothing else is zero, in every kernel that can take the call."""
import pytest
import torch

from test_gpu_cache_attn import E, Problem

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "bf16-ffma", "f32"]
# few rows per sequence and many, with one stream's outputs and two
LENS = [([(300, 1), (140, 2)], 128), ([(300, 70), (140, 60)], 128), ([(300, 2)], 256), ([(300, 70)], 256)]
HEADS, KV = 4, 2


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def problem(lens, d, kind, seed, tree=False):
    """Queries whose first component is 1, so that a key's first component alone can make its score infinite."""
    p = Problem(lens, HEADS, KV, d, 16, torch.float32 if kind == "f32" else torch.bfloat16, tree, seed=seed)
    p.Q[:, :, 0] = 1.0
    return p


def set_keys(p, b, keys, value):
    keys = torch.as_tensor(keys, device="cuda")
    p.K[p.table[b].long()[keys // 16], :, keys % 16, 0] = value


def check(p, O, dead, scale):
    """Against 64 bits, where sequence b's keys in dead[b] are seen by nobody.  Tolerances as in test_gpu_cache_attn."""
    q0 = 0
    for b, (c, n) in enumerate(p.lens):
        key = torch.arange(c + n, device="cuda")
        page = p.table[b].long()[key // 16]
        K, V = (x[page, :, key % 16].double() for x in (p.K, p.V))
        seen = p.seen(b).clone()
        seen[:, dead[b]] = False
        used = seen.any(0)
        for h in range(HEADS):
            k, v = (torch.where(used[:, None], x[:, h * KV // HEADS], 0.0) for x in (K, V))
            q = p.Q[q0:q0 + n, h].double()
            P = torch.softmax((q @ k.t() * scale).masked_fill(~seen, -float("inf")), 1).nan_to_num(0.0)
            ref, size = P @ v, P @ v.abs()
            x = 2 * (p.d + 8) * 2 * E * ((q.abs() @ k.abs().t()) * abs(scale) * seen).amax(1, keepdim=True)
            u = torch.finfo(p.dt).eps / 2
            tol = u * ref.abs() + (x + (c + n + 64) * E + (2.0 ** -8 if p.dt == torch.bfloat16 else 0.0)) * 1.01 * size
            assert bool(((O[q0:q0 + n, h].double() - ref).abs() <= tol).all()), (b, h)
            none = ~seen.any(1)
            assert bool((O[q0:q0 + n, h][none] == 0).all())
        q0 += n


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,d", LENS)
def test_keys_at_minus_infinity(tp, kind, lens, d, sign):
    scale = sign * d ** -0.5
    algo = tp.ALGO_SIMT if kind == "bf16-ffma" else None
    every = [list(range(c + n)) for c, n in lens]
    # some; a whole tile and more, at the beginning or at the end; all
    for dead in ([e[3::7] for e in every], [e[:130] for e in every], [e[100:] for e in every], every):
        p = problem(lens, d, kind, 3)
        for b, keys in enumerate(dead):
            set_keys(p, b, keys, -sign * float("inf"))
        O = p.run(tp, algo, scale=scale)
        assert tp.check_device_status(p.ctx) == tp.OK
        check(p, O, dead, scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,d", LENS)
def test_in_a_tree(tp, kind, lens, d):
    """The same next to keys that are not seen."""
    p = problem(lens, d, kind, 4, tree=True)
    dead = [[i for i in range(c + n) if i % 3 == 1 or i > c] for c, n in lens]
    for b, keys in enumerate(dead):
        set_keys(p, b, keys, -float("inf"))
    O = p.run(tp, tp.ALGO_SIMT if kind == "bf16-ffma" else None)
    check(p, O, dead, d ** -0.5)


@pytest.mark.parametrize("kind", KINDS)
def test_products_past_the_range(tp, kind):
    """All scores are the product of finite numbers past the largest one."""
    p = problem([(200, 3)], 64, kind, 5)
    p.Q[:, :, 0], p.K[..., 0] = 1e30, -1e30
    O = p.run(tp, tp.ALGO_SIMT if kind == "bf16-ffma" else None)
    assert bool((O == 0).all())
