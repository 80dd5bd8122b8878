"""The Newton-Schulz orthogonalisation on the GPU against 64 bits.

Tolerance.  One step is X' = (a - d) X + a lo + (C + dI) X_hi with A and C rounded to fp16: a
rounding is 2^-11 at most and 2^-11/sqrt(3) = 2.8e-4 in the mean of the relative squares.  Near
the end ||A||_F and ||X||_F are about sqrt(p): A's rounding reaches X' through
b + 2cA, a factor of at most 4.8 there, 1.35e-3 of ||X||_F, and C + dI's through X, under
4e-4; a step passes on what it got with a factor below 1 near the end (|f'| <= 0.8 for
singular values in [0.7, 1.2]), so the steps' errors add up to at most
1.4e-3 / sqrt(1 - 0.64) = 2.4e-3.  The output's own rounding to bf16 adds 2^-8/sqrt(3) = 2.3e-3 at
most (1.7e-3 over a spread of values): 3.3e-3 in all, and 5e-3 is allowed for the
2-norm.  Per element: 2^-8 of the element plus eight standard deviations of the rest.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)
TOL = 5e-3


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def reference(G, steps=5, coef=COEF, eps=1e-7):
    a, b, c = coef
    G = G.double()
    out = torch.empty_like(G)
    for i in range(G.shape[0]):
        X = G[i] if G.shape[1] <= G.shape[2] else G[i].t()
        X = X / (torch.linalg.vector_norm(X) + eps)
        for _ in range(steps):
            A = X @ X.t()
            X = a * X + (b * A + c * (A @ A)) @ X
        out[i] = X if G.shape[1] <= G.shape[2] else X.t()
    return out


def check(O, ref):
    O = O.double()
    for i in range(O.shape[0]):
        n = float(ref[i].norm())
        rms = n / ref[i].numel() ** 0.5
        d = O[i] - ref[i]
        assert float(d.norm()) <= TOL * n, (i, float(d.norm()) / n)
        assert bool((d.abs() <= 2.0 ** -8 * ref[i].abs() + 8 * 2.4e-3 * max(rms, float(ref[i].abs().max()) / 4)).all())


def rand(batch, rows, cols, dtype=torch.bfloat16, seed=0, kind="gauss"):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    if kind == "gauss":
        G = torch.randn(batch, rows, cols, generator=g)
    elif kind == "lowrank":  # a few strong directions over weak noise
        k = max(1, min(rows, cols) // 16)
        G = torch.randn(batch, rows, k, generator=g) @ torch.randn(batch, k, cols, generator=g) \
            + 0.01 * torch.randn(batch, rows, cols, generator=g)
    else:  # one strong mean direction
        G = torch.randn(batch, rows, cols, generator=g) + 3.0
    return G.to(dtype).cuda()


def run(tp, G, **kw):
    ctx = tp.OrthoContext(G.shape[1], G.shape[2], G.shape[0], G.dtype, **kw)
    O = tp.orthogonalize(ctx, G)
    assert tp.check_device_status(ctx) == tp.OK
    return O


SHAPES = [  # batch, rows, cols
    (1, 1, 1), (1, 1, 40), (2, 7, 5), (3, 16, 64), (1, 64, 64), (2, 65, 63), (1, 128, 512), (4, 200, 120),
    (1, 256, 256), (1, 257, 1024), (2, 1000, 264), (1, 515, 1003), (5, 300, 300), (1, 1024, 700), (33, 32, 130), (2, 48, 48),
    (3, 17, 300), (1, 90, 90), (2, 700, 112), (1, 128, 129), (1, 130, 127),
    (1, 150, 6000), (2, 5003, 200),  # long and few tiles: the Gram product split
]


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_against_64_bits(tp, batch, rows, cols, dtype):
    G = rand(batch, rows, cols, dtype, seed=rows + cols)
    check(run(tp, G), reference(G))


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(tp, seed):
    import math
    import random
    r = random.Random(2000 + seed)
    size = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))
    rows, cols, batch = size(1, 3000), size(1, 3000), size(1, 12)
    while batch * rows * cols > 4_000_000:
        rows, cols = (rows + 1) // 2, (cols + 1) // 2
    G = rand(batch, rows, cols, r.choice((torch.float32, torch.bfloat16)), seed=seed,
             kind=r.choice(("gauss", "lowrank", "mean")))
    check(run(tp, G), reference(G))


@pytest.mark.parametrize("kind", ["lowrank", "mean"])
@pytest.mark.parametrize("rows,cols", [(256, 640), (640, 256), (384, 384), (4, 5133), (22, 4031), (5827, 34)])
def test_ill_conditioned(tp, rows, cols, kind):
    """Singular values that differ by three orders of magnitude: the small ones keep their directions."""
    G = rand(2, rows, cols, torch.bfloat16, seed=1, kind=kind)
    check(run(tp, G), reference(G))


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_any_magnitude(tp, scale):
    """The norm neither overflows nor underflows (with eps = 0 the scale cancels)."""
    for dtype in (torch.float32, torch.bfloat16):
        for rows, cols in ((96, 160), (300, 200)):
            G = (rand(1, rows, cols, torch.float32, seed=2) * scale).to(dtype)
            check(run(tp, G, eps=0.0), reference(G, eps=0.0))
    # small and ordinary values side by side
    G = rand(1, 160, 200, torch.float32, seed=2)
    G[:, :80] *= scale
    check(run(tp, G, eps=0.0), reference(G, eps=0.0))


@pytest.mark.parametrize("rows,cols", [(80, 96), (200, 264), (264, 200)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_zero_and_non_finite_matrices(tp, rows, cols, bad):
    G = rand(4, rows, cols, seed=3)
    G[1] = 0
    G[2, 3, 4] = bad
    O = run(tp, G)
    ref = reference(G[[0, 3]])
    check(O[[0, 3]], ref)
    assert not bool(O[1].any())
    assert not bool(torch.isfinite(O[2]).all())
    assert not bool(run(tp, torch.zeros_like(G), eps=0.0).any())


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("rows,cols", [(130, 200), (100, 200), (200, 60)])
def test_steps(tp, steps, rows, cols):
    G = rand(2, rows, cols, seed=4)
    check(run(tp, G, steps=steps), reference(G, steps))


def test_other_coefficients(tp):
    """The convergent cubic s (3 - s^2)/2 and a quintic that converges to 1."""
    G = rand(1, 100, 300, seed=5)
    G2 = rand(1, 300, 160, seed=5)
    for coef in ((1.5, -0.5, 0.0), (1.875, -1.25, 0.375)):
        check(run(tp, G, steps=12, coefficients=coef), reference(G, 12, coef))
        check(run(tp, G2, steps=12, coefficients=coef), reference(G2, 12, coef))
    # too many steps for Q in fp16's range: the steps on X itself
    check(run(tp, G, steps=20, coefficients=(1.875, -1.25, 0.375)), reference(G, 20, (1.875, -1.25, 0.375)))


def test_same_bits_again_in_a_batch_and_on_another_stream(tp):
    G = rand(3, 300, 520, seed=6)
    O = run(tp, G)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run(tp, G)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(O, again)


def test_two_dimensions_guards_and_offset_views(tp):
    """An output inside a larger buffer: its neighbours stay as they were, odd sizes and bases too."""
    for rows, cols in ((90, 104), (90, 103)):
        G = rand(1, rows, cols, seed=7)
        ctx = tp.OrthoContext(rows, cols, dtype=G.dtype)
        room = torch.full((rows * cols + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        at = 8 if cols % 8 == 0 else 3
        O = room[at:at + rows * cols].view(rows, cols)
        tp.orthogonalize(ctx, G[0], O)
        check(O[None], reference(G))
        assert bool((room[:at] == 7).all()) and bool((room[at + rows * cols:] == 7).all())
        src = torch.empty(rows * cols + 1, dtype=G.dtype, device="cuda")
        src[1:] = G.reshape(-1)
        assert torch.equal(tp.orthogonalize(ctx, src[1:].view(rows, cols)), O)


def test_captured_and_replayed(tp):
    G = rand(2, 128, 192, seed=8)
    ctx = tp.OrthoContext(128, 192, 2)
    O = torch.empty_like(G)
    tp.orthogonalize(ctx, G, O)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tp.orthogonalize(ctx, G, O)
    G.copy_(rand(2, 128, 192, seed=9))
    g.replay()
    torch.cuda.synchronize()
    check(O, reference(G))


@pytest.mark.parametrize("rows,cols", [(96, 200), (300, 200), (70, 33)])
def test_in_place(tp, rows, cols):
    G = rand(2, rows, cols, seed=10)
    want = run(tp, G)
    ctx = tp.OrthoContext(rows, cols, 2)
    assert tp.orthogonalize(ctx, G, G) is G
    assert torch.equal(G, want)


def test_a_batch_past_32_bits(tp):
    """65 matrices of 4096 x 8192, 2.2e9 elements: the last one like the first."""
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    n, r, c = 65, 4096, 8192
    G = torch.empty(n, r, c, dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        G[i] = torch.randn(r, c, device="cuda")
    O = run(tp, G)
    for i in (0, n - 1):  # (alone it may round differently: other tiles, other orders)
        check(O[i:i + 1], reference(G[i:i + 1]))


def test_empty_batch(tp):
    ctx = tp.OrthoContext(8, 8, 0)
    assert tp.orthogonalize(ctx, torch.empty(0, 8, 8, dtype=torch.bfloat16, device="cuda")).shape == (0, 8, 8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(100, 3000), (1100, 1000)])
@pytest.mark.parametrize("scale", [2.0 ** 126, 2.0 ** 100, 2.0 ** 47, 2.0 ** 45, 2.0 ** -55, 2.0 ** -57, 2.0 ** -115,
                                   2.0 ** -130, 2.0 ** -143])
def test_norms_at_the_ends_of_the_range(tp, rows, cols, scale, dtype):
    """A million of the largest numbers (the sum of their squares is past fp32 in any one unit that also
    holds the middle ones), and matrices wholly of subnormal ones, of which 2^-143 leaves fp32 six bits,
    and bf16 none."""
    G = rand(1, rows, cols, torch.float32, seed=11).clamp_(-3, 3)
    if scale == 2.0 ** 126:
        G = torch.sign(G) * (2 + G.abs() / 3)  # up to 3 * 2^126
    G = (G.double() * scale).to(dtype)
    assert bool(torch.isfinite(G).all())
    if not bool(G.any()):
        assert not bool(run(tp, G, eps=0.0).any())
        return
    check(run(tp, G, eps=0.0), reference(G, eps=0.0))


def test_norm_of_all_kinds_of_values_at_once(tp):
    """Large, ordinary and tiny values in one matrix, in every unit of the sum."""
    for hi, lo in ((2.0 ** 60, 1.0), (2.0 ** 50, 2.0 ** 40), (1.0, 2.0 ** -60), (2.0 ** -50, 2.0 ** -58), (2.0 ** 120, 2.0 ** -140)):
        for rows, cols in ((64, 600), (300, 200)):
            G = rand(1, rows, cols, torch.float32, seed=12).double()
            G[:, : rows // 2] *= hi
            G[:, rows // 2:] *= lo
            G = G.float()
            keep = slice(0, rows // 2)
            O, ref = run(tp, G, eps=0.0), reference(G, eps=0.0)
            # (rows of the smaller scale are beyond the condition that the iterates hold)
            if hi / lo <= 2.0 ** 10:
                check(O, ref)
            else:
                check(O[:, keep], ref[:, keep])


@pytest.mark.parametrize("steps,coef", [(5, COEF), (6, COEF), (7, COEF), (8, COEF), (9, (3.0, -3.2, 1.2)), (6, (3.0, -3.2, 1.2)),
                                        (9, (2.0, -1.5, 0.5)), (12, (2.0, -1.5, 0.5)), (10, (1.875, -1.25, 0.375)),
                                        (13, (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("rows,cols", [(120, 706), (16, 300), (600, 50), (200, 300)])
def test_many_steps_on_strong_directions_over_noise(tp, rows, cols, steps, coef):
    """Small singular values grow by a factor of up to a^steps (500 to 40000 here) while the strong ones stay:
    what a step does to the small ones may not be lost in the roundings of the large ones."""
    for dtype in (torch.float32, torch.bfloat16):
        for k, strong in ((1, 100.0), (4, 30.0)):
            g = torch.Generator(device="cpu")
            g.manual_seed(13)
            G = torch.randn(2, rows, k, generator=g) @ torch.randn(2, k, cols, generator=g) * (strong / min(rows, cols) ** 0.5)
            G = (G + 0.01 * torch.randn(2, rows, cols, generator=g)).to(dtype).cuda()
            check(run(tp, G, steps=steps, coefficients=coef), reference(G, steps, coef))
        G = rand(2, rows, cols, dtype, seed=14, kind="lowrank")
        check(run(tp, G, steps=steps, coefficients=coef), reference(G, steps, coef))
