"""The vocabulary cross entropy on the GPU against a plain implementation in 64 bits.

Tolerances, per element and derived from the arithmetic:
- a logit is a sum of h exact products, accumulated in fp32 with an error of at most
  (h + 8) 2^-23 sum_k |x_k w_k| (2^-23, not 2^-24, allows an accumulator that truncates);
  call the largest of a token e.  loss and lse move by at most 2e and e, plus 2^-20 of
  their terms for the exponentials, the join and the logarithm;
- an fp32 operand a is a sum of three bf16 numbers, whose steps are 2^-133 at the least: where
  that cuts a short (below 2^-110) its sum is off by at most half a step, 2^-134.  With
  x + d and w + f for x and w, x w moves by |d w| + |x f| + |d f|, so a logit by at most
  2^-134 (sum |x_k| + sum |w_k| + h 2^-134), which e takes in (for sums up to 2^100 it is under
  2^-33, nothing);
- dS = (p - 1[y]) g: p moves by a factor of at most exp(2e) (1 + 2^-20), then one rounding
  to the dtype, u = eps/2 relative;
- a probability below 2^-126, the smallest normal fp32 number, comes out of the exponential
  as zero, and so may a dS or a sum below it: 2^-126 absolute, three times;
- dX and dW are sums of n products of dS: the errors of dS times |W| or |X|, the
  accumulation n 2^-23, and one rounding of the result.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

IGN = -100


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def make(T, h, V, dtype=torch.bfloat16, seed=0, ignored=0.0, scale=1.0, ignore_index=IGN):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    X = torch.randn(T, h, generator=g) * scale
    W = torch.randn(V, h, generator=g) * (1.3 / math.sqrt(h))
    y = torch.randint(0, V, (T,), generator=g)
    drop = torch.rand(T, generator=g) < ignored
    y = torch.where(drop, torch.full_like(y, ignore_index), y)
    dl = torch.rand(T, generator=g) * 2 / max(T, 1)
    return X.to(dtype).cuda(), W.to(dtype).cuda(), y.cuda(), dl.cuda()


def reference(X, W, y, dl, ignore_index=IGN):
    X, W, dl = X.double(), W.double(), dl.double()
    S = X @ W.t()
    lse = torch.logsumexp(S, 1)
    ok = y != ignore_index
    at = torch.where(ok, y, 0)[:, None]
    loss = torch.where(ok, lse - S.gather(1, at)[:, 0], 0.0)
    P = torch.exp(S - lse[:, None])
    P.scatter_add_(1, at, -ok.double()[:, None])
    g = torch.where(ok, dl, 0.0)[:, None]
    dS = torch.where(g != 0, P * g, 0.0)
    return {"S": S, "lse": lse, "loss": loss, "dS": dS, "dX": dS @ W, "dW": dS.t() @ X}


def check(X, W, y, dl, loss, lse, grads, ref):
    T, h = X.shape
    V = W.shape[0]
    dt = X.dtype
    u = torch.finfo(dt).eps / 2
    Xa, Wa = X.double().abs(), W.double().abs()
    e = (h + 8) * 2.0 ** -23 * (Xa @ Wa.t()).amax(1)
    if dt == torch.float32:
        e = e + 2.0 ** -134 * (Xa.sum(1) + Wa.sum(1).amax() + h * 2.0 ** -134)
    small = 2.0 ** -20 * (ref["S"].abs().amax(1) + math.log(V) + 1)
    assert bool(((lse.double() - ref["lse"]).abs() <= e + small).all())
    assert bool(((loss.double() - ref["loss"]).abs() <= 2 * e + 2 * small).all())
    if grads is None:
        return
    # p's own error: relative on p, also where p - 1 cancels, to nothing with V = 1: lse and the
    # recomputed logit are then two roundings of the same sum, up to 2e apart, and dS is
    # (exp(2e) - 1) g instead of 0
    P = torch.exp(ref["S"] - ref["lse"][:, None])
    g = torch.where(y != IGN, dl.double(), 0.0)[:, None]
    dp = torch.expm1(2 * e + small)[:, None] * P * g.abs()
    err_s = dp + (u + 2.0 ** -22) * (ref["dS"].abs() + dp) + 2 * 2.0 ** -126
    for name, other, left in (("dX", Wa, False), ("dW", Xa, True)):
        if grads[name] is None:
            continue
        a = ref["dS"].abs().t() if left else ref["dS"].abs()
        s = err_s.t() if left else err_s
        n = a.shape[1]
        tol = (s @ other) + (n + 64) * 2.0 ** -23 * (a @ other)
        tol = tol + u * (ref[name].abs() + tol) + 2.0 ** -126
        bad = (grads[name].double() - ref[name]).abs() > tol
        assert not bool(bad.any()), (name, int(bad.sum()))


def run(tp, X, W, y, dl, **kw):
    ctx = tp.XentContext(X.shape[0], X.shape[1], W.shape[0], X.dtype, **kw)
    loss = tp.xent_forward(ctx, X, W, y)
    grads = tp.xent_backward(ctx, dl)
    assert tp.check_device_status(ctx) == tp.OK
    return ctx, loss, grads


SHAPES = [  # T, h, V: one token, ragged tiles in every dimension, vocabulary of one row, long rows
    (1, 8, 1), (1, 64, 17), (3, 72, 513), (31, 128, 255), (128, 256, 512), (129, 264, 1025), (256, 512, 4096),
    (300, 200, 3001), (257, 1000, 777), (1000, 96, 2049), (5, 4096, 8191), (2, 8192, 130),
    (1, 24, 5000), (2, 1000, 333), (4, 264, 20000), (7, 40, 61), (8, 8192, 700), (8, 64, 3), (9, 200, 999), (16, 4096, 300),
    (20, 104, 5003), (32, 1024, 77), (32, 24, 6000), (33, 64, 500),  # a pass over W
    (40, 64, 30011), (6000, 72, 100),  # K of dX and of dW long, few tiles: split
]


@pytest.mark.parametrize("T,h,V", SHAPES)
def test_bf16_against_64_bits(tp, T, h, V):
    X, W, y, dl = make(T, h, V, seed=T + h + V, ignored=0.2)
    ctx, loss, grads = run(tp, X, W, y, dl)
    check(X, W, y, dl, loss, ctx.lse, grads, reference(X, W, y, dl))


@pytest.mark.parametrize("T,h,V", [(1, 1, 1), (3, 5, 7), (64, 33, 1000), (130, 256, 777), (300, 770, 2500),
                                   (17, 40, 20011), (5000, 36, 90), (4100, 9, 33),
                                   (1, 4100, 700), (5, 130, 3000), (8, 8192, 50)])
def test_f32_against_64_bits(tp, T, h, V):
    X, W, y, dl = make(T, h, V, torch.float32, seed=T + h + V, ignored=0.2)
    ctx, loss, grads = run(tp, X, W, y, dl)
    check(X, W, y, dl, loss, ctx.lse, grads, reference(X, W, y, dl))


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(tp, seed):
    """Sizes over their whole range (logarithmically), types, pieces and ignored shares at random."""
    import random
    r = random.Random(1000 + seed)
    size = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))
    f32 = r.random() < 0.4
    T, V = size(1, 3000), size(1, 12000)
    h = size(1, 700) if f32 else 8 * size(1, 300)
    while T * V > 6_000_000:
        T, V = (T + 1) // 2, (V + 1) // 2
    X, W, y, dl = make(T, h, V, torch.float32 if f32 else torch.bfloat16, seed=seed, ignored=r.choice((0, 0.3, 0.9)))
    ctx, loss, grads = run(tp, X, W, y, dl, piece=r.choice((0, 0, 8 * size(8, 400))))
    check(X, W, y, dl, loss, ctx.lse, grads, reference(X, W, y, dl))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("piece", [8, 64, 520, 1024, 4096])
def test_pieces(tp, piece, dtype):
    """Any division of the vocabulary gives the same loss and, within tolerance, gradients."""
    X, W, y, dl = make(70, 128, 1300, dtype, seed=piece, ignored=0.3)
    ref = reference(X, W, y, dl)
    ctx, loss, grads = run(tp, X, W, y, dl, piece=piece)
    check(X, W, y, dl, loss, ctx.lse, grads, ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ffma_path(tp, dtype):
    X, W, y, dl = make(100, 192, 1111, dtype, seed=3, ignored=0.1)
    ref = reference(X, W, y, dl)
    for piece in (0, 512):
        ctx, loss, grads = run(tp, X, W, y, dl, algo=tp.ALGO_SIMT, piece=piece)
        check(X, W, y, dl, loss, ctx.lse, grads, ref)


def test_every_token_ignored_and_ignore_index_inside_the_vocabulary(tp):
    X, W, y, dl = make(40, 64, 300, seed=1)
    ctx, loss, grads = run(tp, X, W, torch.full_like(y, IGN), dl)
    assert not bool(loss.any()) and not bool(grads["dX"].any()) and not bool(grads["dW"].any())
    y[::3] = 7
    ctx, loss, grads = run(tp, X, W, y, dl, ignore_index=7)
    ref = reference(X, W, y, dl, 7)
    assert not bool(loss[::3].any())
    assert torch.allclose(loss.double(), ref["loss"], atol=1e-4)
    u = 2.0 ** -8  # coarse: the sharp bounds are checked above
    assert float((grads["dX"].double() - ref["dX"]).norm() / ref["dX"].norm()) < 2 * u


def test_large_logits_and_small_probabilities(tp):
    """Logits of several hundred: the maximum is subtracted before any exponential."""
    X, W, y, dl = make(64, 128, 1000, seed=2, scale=100.0)
    ctx, loss, grads = run(tp, X, W, y, dl)
    ref = reference(X, W, y, dl)
    assert float(ref["S"].abs().max()) > 300
    check(X, W, y, dl, loss, ctx.lse, grads, ref)


def test_non_finite_tokens_stay_alone(tp):
    X, W, y, dl = make(300, 64, 700, seed=4)
    X[5, 3] = float("nan")
    X[290, 1] = float("inf")
    y[7] = IGN
    X[7] = float("nan")  # an ignored token's logits reach neither its loss nor dW
    ctx, loss, grads = run(tp, X, W, y, dl)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[5, 7, 290]] = False
    assert not bool(torch.isfinite(loss[[5, 290]]).any())
    assert float(loss[7]) == 0.0 and not bool(grads["dX"][7].any())
    ref = reference(X[keep], W, y[keep], dl[keep])
    assert torch.allclose(loss[keep].double(), ref["loss"], atol=1e-4)
    assert bool(torch.isfinite(grads["dX"][keep]).all())


def test_a_target_outside_the_vocabulary_is_reported(tp):
    X, W, y, dl = make(50, 64, 100, seed=5)
    for bad in (100, -1, 2 ** 40):
        y2 = y.clone()
        y2[11] = bad
        ctx = tp.XentContext(50, 64, 100, X.dtype)
        loss = tp.xent_forward(ctx, X, W, y2)
        assert tp.check_device_status(ctx) == tp.ERR_INVALID_ARG
        y3 = y.clone()
        y3[11] = IGN
        want = tp.xent_forward(ctx, X, W, y3)
        assert tp.check_device_status(ctx) == tp.OK
        assert torch.equal(loss, want)


def test_outputs_left_out_and_guards_kept(tp):
    """A frozen head or body: the other gradient has the same bits; nothing outside an output is written."""
    X, W, y, dl = make(130, 136, 1001, seed=6, ignored=0.1)
    ctx, loss, grads = run(tp, X, W, y, dl, piece=512)
    only = tp.xent_backward(ctx, dl, need_dW=False)
    assert only["dW"] is None and torch.equal(only["dX"], grads["dX"])
    only = tp.xent_backward(ctx, dl, need_dX=False)
    assert only["dX"] is None and torch.equal(only["dW"], grads["dW"])
    room_x = torch.full((132, 136), 7.0, dtype=X.dtype, device="cuda")
    room_w = torch.full((1003, 136), 7.0, dtype=X.dtype, device="cuda")
    tp.xent_backward(ctx, dl, dX=room_x[1:131], dW=room_w[1:1002])
    assert torch.equal(room_x[1:131], grads["dX"]) and torch.equal(room_w[1:1002], grads["dW"])
    assert bool((room_x[[0, 131]] == 7).all()) and bool((room_w[[0, 1002]] == 7).all())


def test_same_bits_again_and_on_another_stream(tp):
    X, W, y, dl = make(513, 256, 5000, seed=7)
    ctx, loss, grads = run(tp, X, W, y, dl, piece=1536)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ctx2, loss2, grads2 = run(tp, X, W, y, dl, piece=1536)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(loss, loss2) and torch.equal(ctx.lse, ctx2.lse)
    assert torch.equal(grads["dX"], grads2["dX"]) and torch.equal(grads["dW"], grads2["dW"])


@pytest.mark.parametrize("T", [1, 5, 200])
def test_captured_and_replayed(tp, T):
    X, W, y, dl = make(T, 128, 3000, seed=8)
    ctx, loss, grads = run(tp, X, W, y, dl, piece=1024)
    out = torch.empty_like(loss)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tp.xent_forward(ctx, X, W, y, out)
        tp.xent_backward(ctx, dl, dX, dW)
    X2, _, y2, _ = make(T, 128, 3000, seed=9)
    X.copy_(X2)
    y.copy_(y2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    check(X, W, y, dl, out, ctx.lse, {"dX": dX, "dW": dW}, reference(X, W, y, dl))


def test_f32_at_the_end_of_its_range(tp):
    """The largest fp32 numbers do not become infinite in bf16 parts: X next to 2^128 times W small."""
    X, W, y, dl = make(40, 64, 200, torch.float32, seed=14)
    X[:, 0], W[:, 0] = torch.finfo(torch.float32).max, W[:, 0] * 1e-38
    X[3, 5], W[:, 5] = -torch.finfo(torch.float32).max, 0.0
    ctx, loss, grads = run(tp, X, W, y, dl)
    ref = reference(X, W, y, dl)
    check(X, W, y, dl, loss, ctx.lse, {"dX": grads["dX"], "dW": None}, ref)
    assert bool(torch.isfinite(grads["dW"][:, 1:5]).all())


@pytest.mark.parametrize("T,h,V", [(3, 36, 500), (50, 36, 500), (50, 33, 70)])
def test_f32_on_any_element(tp, T, h, V):
    """fp32 inputs and outputs that start on 4 bytes only."""
    def shifted(x):
        room = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        room[1:] = x.reshape(-1)
        return room[1:].view(x.shape)

    X, W, y, dl = make(T, h, V, torch.float32, seed=T)
    X, W = shifted(X), shifted(W)
    ctx = tp.XentContext(T, h, V, X.dtype)
    loss = tp.xent_forward(ctx, X, W, y)
    dX, dW = shifted(torch.empty_like(X)), shifted(torch.empty_like(W))
    grads = tp.xent_backward(ctx, dl, dX, dW)
    check(X, W, y, dl, loss, ctx.lse, grads, reference(X, W, y, dl))


@pytest.mark.parametrize("T", [1, 3, 16])
def test_a_vocabulary_past_32_bits(tp, T):
    """W and dW of 2.2e9 elements: rows at the far end count like the others."""
    h, V = 8192, 270000
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    W = torch.empty(V, h, dtype=torch.bfloat16, device="cuda")
    for i in range(0, V, 30000):
        W[i:i + 30000] = torch.randn(30000, h, generator=g, device="cuda") * 0.01
    X = torch.randn(T, h, generator=g, device="cuda").bfloat16()
    y = torch.full((T,), V - 1, device="cuda")
    y[T // 2] = V - 4097
    dl = torch.ones(T, device="cuda")
    ctx = tp.XentContext(T, h, V, X.dtype)
    loss = tp.xent_forward(ctx, X, W, y)
    grads = tp.xent_backward(ctx, dl)
    assert tp.check_device_status(ctx) == tp.OK
    S = torch.cat([X.double() @ W[i:i + 30000].double().t() for i in range(0, V, 30000)], 1)
    lse = torch.logsumexp(S, 1)
    assert torch.allclose(loss.double(), lse - S.gather(1, y[:, None])[:, 0], rtol=0, atol=1e-3)
    P = torch.exp(S - lse[:, None])
    P.scatter_add_(1, y[:, None], -torch.ones_like(P[:, :1]))
    u = 2.0 ** -8
    for rows in (slice(0, 1000), slice(V - 5000, V)):
        ref = P[:, rows].t() @ X.double()
        # one rounding of dS and one of dW, and the logits' error of 1e-3 in p
        tol = (2.1 * u + 2e-3) * (P[:, rows].abs().t() @ X.double().abs())
        assert bool(((grads["dW"][rows].double() - ref).abs() <= tol + 1e-30).all())
    dX = sum(P[:, i:i + 30000] @ W[i:i + 30000].double() for i in range(0, V, 30000))
    assert float((grads["dX"].double() - dX).norm()) <= 2 * u * float(dX.norm())


def test_equal_weights_leave_no_bias(tp):
    """The same dloss for every token, half way between two bf16 numbers: rounding dS token by
    token would move every target's term the same way, by 2^-9 to 2^-8 of it.  With T
    terms rounded apart the mean error is at most 2^-8 / sqrt(3 T) in the mean of squares,
    1e-4 for T = 512; 2^-10 is nine times that."""
    X, W, y, _ = make(512, 256, 4000, seed=11)
    dl = torch.full((512,), (1 + 2.0 ** -8) / 512, device="cuda")
    for piece in (0, 2048):
        ctx, loss, grads = run(tp, X, W, y, dl, piece=piece)
        ref = reference(X, W, y, dl)
        check(X, W, y, dl, loss, ctx.lse, grads, ref)
        for n in ("dX", "dW"):
            along = float((grads[n].double() * ref[n]).sum() / (ref[n] * ref[n]).sum())
            assert abs(along - 1) < 2.0 ** -10, (n, along)


@pytest.mark.parametrize("T,h,V", [(8192, 4096, 2560), (2048, 8192, 9000), (300, 4096, 2000)])
def test_long_sums_leave_no_bias(tp, T, h, V):
    """What is asked of the loss of bf16 inputs: within 1e-6 of itself, over all tokens, at lengths
    where an accumulator that truncates at every 16 products shrinks a logit by about
    2^-26 h / 16 of itself, 3.8e-6 for h = 4096."""
    X, W, y, _ = make(T, h, V, seed=17)
    X = (X.float() + torch.linspace(0, 4, T, device="cuda")[:, None] * W[y].float()).bfloat16()  # towards the target
    ctx = tp.XentContext(T, h, V, torch.bfloat16)
    loss = tp.xent_forward(ctx, X, W, y).double()
    ref = reference(X, W, y, torch.zeros(T, device="cuda"))["loss"]
    assert float((loss - ref).norm() / ref.norm()) <= 1e-6


def test_workspace_is_left_ready_for_the_next_call(tp):
    """Calls of different kinds share one workspace, with other workspace contents between them."""
    X, W, y, dl = make(4, 128, 700, seed=12)
    ctx = tp.XentContext(4, 128, 700, X.dtype)
    want = tp.xent_forward(ctx, X, W, y).clone()
    for _ in range(3):
        tp.xent_backward(ctx, dl)
        ctx.workspace[1024:] = 255
        assert torch.equal(tp.xent_forward(ctx, X, W, y), want)


def test_a_context_on_its_tensors_device_only(tp):
    X, W, y, dl = make(4, 64, 50, seed=13)
    ctx = tp.XentContext(4, 64, 50, X.dtype)
    with pytest.raises(ValueError):
        tp.xent_forward(ctx, X.cpu(), W, y)
    with pytest.raises(ValueError):
        tp.xent_backward(ctx, dl)  # no forward yet
    with pytest.raises(ValueError):
        tp.xent_forward(ctx, X, W, y.int())
    with pytest.raises(ValueError):
        tp.xent_forward(ctx, X, W.t().contiguous().t(), y)
    with pytest.raises(tp.TpmlpError):
        tp.xent_forward(tp.XentContext(4, 60, 50, X.dtype), X[:, :60].contiguous(), W[:, :60].contiguous(), y)


def test_no_tokens(tp):
    W = torch.randn(100, 64, device="cuda").bfloat16()
    X = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    ctx = tp.XentContext(0, 64, 100, torch.bfloat16)
    loss = tp.xent_forward(ctx, X, W, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert loss.shape == (0,)
    grads = tp.xent_backward(ctx, loss)
    assert grads["dX"].shape == (0, 64) and not bool(grads["dW"].any())


def test_gradient_against_differences(tp):
    """dX in fp32 against central differences of the 64-bit loss along random directions: the
    third-order term is far below, the loss is exact to 64 bits."""
    X, W, y, dl = make(20, 48, 90, torch.float32, seed=10)
    _, _, grads = run(tp, X, W, y, dl)

    def total(Xd, Wd):
        S = Xd @ Wd.t()
        return float((dl.double() * (torch.logsumexp(S, 1) - S.gather(1, y[:, None])[:, 0])).sum())

    for k in range(3):
        dx, dw = torch.randn_like(X).double(), torch.randn_like(W).double()
        eps = 1e-5
        num = (total(X.double() + eps * dx, W.double() + eps * dw)
               - total(X.double() - eps * dx, W.double() - eps * dw)) / (2 * eps)
        ana = float((grads["dX"].double() * dx).sum() + (grads["dW"].double() * dw).sum())
        scale = float((grads["dX"].double() * dx).abs().sum() + (grads["dW"].double() * dw).abs().sum())
        assert abs(num - ana) <= 1e-5 * scale + 1e-9


@pytest.mark.parametrize("masked", ["ignored, dloss 0", "ignored, another dloss", "dloss 0", "outside", "nan dloss"])
@pytest.mark.parametrize("n", [1, 100, 300])
def test_equal_weights_after_masked_tokens_leave_no_bias(tp, masked, n):
    """The bound of the test above where the first n tokens have no part in the loss: what their
    dloss holds decides nothing.  Of 512 - n >= 212 tokens the mean error is at most
    2^-8 / sqrt(3 * 212) in the mean of squares, 1.6e-4."""
    X, W, y, _ = make(512, 256, 4000, seed=11)
    dl = torch.full((512,), (1 + 2.0 ** -8) / 512, device="cuda")
    if masked in ("dloss 0", "ignored, dloss 0"):
        dl[:n] = 0
    if masked == "ignored, another dloss":
        dl[:n] = 1.3
    if masked == "nan dloss":
        dl[:n] = float("nan")
    y[:n] = y[:n] if masked == "dloss 0" else IGN
    y_in = y.clone()
    if masked == "outside":
        y_in[:n] = 4000
    for piece in (0, 2048):
        ctx = tp.XentContext(512, 256, 4000, X.dtype, piece=piece)
        loss = tp.xent_forward(ctx, X, W, y_in)
        grads = tp.xent_backward(ctx, dl)
        assert tp.check_device_status(ctx) == (tp.ERR_INVALID_ARG if masked == "outside" else tp.OK)
        ref = reference(X, W, y, dl)
        check(X, W, y, torch.where(y == IGN, 0.0, dl), loss, ctx.lse, grads, ref)
        for name in ("dX", "dW"):
            along = float((grads[name].double() * ref[name]).sum() / (ref[name] * ref[name]).sum())
            assert abs(along - 1) < 2.0 ** -10, (name, along)


@pytest.mark.parametrize("first", [1e-30, 1e30, 3e38])
def test_weights_far_apart(tp, first):
    """The first token's weight next to ordinary ones: neither it nor they leave fp32's range."""
    X, W, y, dl = make(40, 64, 300, seed=15)
    dl[0] = first
    ctx, loss, grads = run(tp, X, W, y, dl)
    ref = reference(X, W, y, dl)
    if first > 1e31:  # dW adds terms of 3e38 up to more than fp32 holds
        grads = {"dX": grads["dX"][1:], "dW": None}
        X, y, dl, loss, lse = X[1:], y[1:], dl[1:], loss[1:], ctx.lse[1:]
        check(X, W, y, dl, loss, lse, grads, reference(X, W, y, dl))
    else:
        check(X, W, y, dl, loss, ctx.lse, grads, ref)


def rows_of_kind(kind, T, h, V, dtype, seed):
    """X and W where the sum of a logit is exact, sparse, padded, or all of one sign."""
    X, W, y, dl = make(T, h, V, torch.float32, seed=seed)
    r = torch.arange(T, device="cuda")
    if kind == "one-hot":
        X = torch.zeros_like(X)
        X[r, (r * 37 + 5) % h] = 64.0
    elif kind == "sparse":
        X = torch.where((r[:, None] * 7 + torch.arange(h, device="cuda")) % 97 == 0, 9 * X, 0.0)
    elif kind == "padded":
        X[:, 64:] = 0
        X *= 8
    elif kind == "one sign":
        X, W = X.abs(), W.abs() / math.sqrt(h)
    elif kind == "towards the target":
        X = X + 4 * W[y]
    return X.to(dtype), W.to(dtype), y, dl


@pytest.mark.parametrize("dtype,h", [(torch.bfloat16, 2048), (torch.bfloat16, 4096), (torch.bfloat16, 8192),
                                     (torch.float32, 256), (torch.float32, 4096)])
@pytest.mark.parametrize("T,V", [(7, 1500), (100, 1500), (600, 2000), (2500, 9000)])
@pytest.mark.parametrize("kind", ["dense", "one-hot", "sparse", "padded", "one sign", "towards the target"])
def test_logits_of_every_kind_of_row(tp, kind, T, V, dtype, h):
    """lse of every token, and the losses' error over all tokens, against 64 bits.

    A logit S comes from accumulations of n products, 2048 (bf16) or 256 (fp32) at the most, that are
    cut off at every step of 16 in which a product is not zero, by at most an ulp of the partial
    sum, half of one on average: at most `steps` 2^-24 of sum |x w| for terms of one sign (the
    partial sum is half the whole on average), and a quarter of `steps` 2^-24 of S for independent
    terms, up to 1.3 times that where they lean one way (1.5 is taken).  The sum of the ranges, the
    difference to the maximum and the logarithm round h / n + 4 times by 2^-24; fp32 leaves out
    products of parts of 2^-22.  The exponentials, their sum and the logarithm leave 2^-21 of
    their own (and of lse and log V in lse)."""
    X, W, y, dl = rows_of_kind(kind, T, h, V, dtype, seed=T + h)
    ctx = tp.XentContext(T, h, V, dtype)
    loss = tp.xent_forward(ctx, X, W, y)
    assert tp.check_device_status(ctx) == tp.OK
    ref = reference(X, W, y, dl)
    n = min(2048 if dtype == torch.bfloat16 else 256, h)
    steps = {"one-hot": 0, "sparse": n / 97 + 1, "padded": 4}.get(kind, n / 16)
    roundings = h / n + 4 + (4 if dtype == torch.float32 else 0)
    size = (X.double().abs() @ W.double().abs().t()).amax(1)
    tol = (steps + roundings) * 2.0 ** -24 * size + 2.0 ** -21 * (ref["lse"].abs() + math.log(V))
    assert bool(((ctx.lse.double() - ref["lse"]).abs() <= tol).all())
    both = ref["S"].abs().amax(1) + ref["S"].gather(1, y[:, None])[:, 0].abs()
    tol = ((steps if kind == "one sign" else 1.5 * steps / 4) + roundings) * 2.0 ** -24 * both + 2.0 ** -21
    assert float((loss.double() - ref["loss"]).norm()) <= float(tol.norm())


def certain(T, h, V, dtype):
    """Tokens whose target's logit (270) is more than 100 above every other, whose exponentials are
    zero in fp32."""
    X, W, y, dl = make(T, h, V, torch.float32, seed=T + h + V)
    W = (W / W.norm(dim=1, keepdim=True)).to(dtype)
    X = (270 * W[y].float()).to(dtype)
    S = X.double() @ W.double().t()
    others = S.scatter(1, y[:, None], -float("inf")).amax(1)
    assert bool((S.gather(1, y[:, None])[:, 0] - others > 100).all())
    return X, W, y, dl


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,h,V", [(1, 256, 300), (5, 1024, 3000), (9, 256, 300), (100, 1000, 2000), (333, 2056, 20000),
                                   (2500, 2048, 9000), (2500, 4096, 9000)])
def test_certain_tokens_have_no_loss(tp, T, h, V, dtype):
    """The sum of exponentials is the maximum's own term, exactly 1, and lse the target's logit."""
    X, W, y, dl = certain(T, h, V, dtype)
    ctx = tp.XentContext(T, h, V, dtype)
    assert not bool(tp.xent_forward(ctx, X, W, y).any())
    assert tp.check_device_status(ctx) == tp.OK


@pytest.mark.parametrize("T", [3, 40, 300])
def test_logits_at_the_end_of_fp32(tp, T):
    """Logits of either sign up to 2^127.5: 1.44 times the maximum would not be a number any more."""
    h, V = 64, 600
    X, W, y, dl = make(T, h, V, seed=16)
    X[:, 0], W[:, 0] = 2.0 ** 100, 0.0
    W[V // 2, 0], W[V // 2 + 1, 0] = 1.375 * 2.0 ** 27, -1.375 * 2.0 ** 27  # 2^127.46 and its negative
    y[:] = V // 2
    y[1::2] = V // 2 + 1
    ctx = tp.XentContext(T, h, V, torch.bfloat16)
    loss = tp.xent_forward(ctx, X, W, y)
    top = 1.375 * 2.0 ** 127
    assert bool((ctx.lse == top).all())
    assert not bool(loss[::2].any()) and bool((loss[1::2] == float("inf")).all())  # 2^128.5 is past fp32


def own_bits(tp, T, h, V, dtype, **kw):
    """p - 1 of a token that is certain of its target is exactly 0 if the backward pass computes the
    same bits for the target's logit, which is lse; else it is an ulp of 270 or more."""
    X, W, y, dl = certain(T, h, V, dtype)
    _, _, grads = run(tp, X, W, y, dl, **kw)
    assert not bool(grads["dX"].any()) and not bool(grads["dW"].any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,h,V", [
    (9, 256, 300), (100, 1000, 2000), (128, 2048, 12000), (200, 4096, 1500), (600, 8192, 2000), (1300, 1032, 9000),
    (2500, 2048, 9000), (2500, 4096, 9000), (4000, 200, 70), (4000, 520, 3000), (333, 2056, 20000)])
def test_both_passes_compute_the_same_logits(tp, T, h, V, dtype):
    own_bits(tp, T, h, V, dtype)
    own_bits(tp, T, h, V, dtype, piece=1024)


def check_confident(tp, T, h, V, dtype, **kw):
    """Tokens fairly sure of their target (1 - p from 1e-6 to 1e-2), every element.  The logits of
    both passes are the same, with errors of at most e (see above) of the exact ones, so p
    is a softmax of logits that are off by e: p moves by p (1 - p) (exp(2 e) - 1).  lse is rounded by
    2^-24 of itself, and 2^-23 of the largest logit is taken, with 2^-21 for the exponentials and the
    logarithm, which p - 1 moves by however small it is."""
    X, W, y, dl = make(T, h, V, torch.float32, seed=T + h)
    X = 0.3 * X + torch.linspace(9, 13, T, device="cuda")[:, None] * W[y]
    X, W = X.to(dtype), W.to(dtype)
    ctx, loss, grads = run(tp, X, W, y, dl, **kw)
    ref = reference(X, W, y, dl)
    Xa, Wa = X.double().abs(), W.double().abs()
    e = (h + 8) * 2.0 ** -23 * (Xa @ Wa.t()).amax(1)
    P = torch.exp(ref["S"] - ref["lse"][:, None])
    rest = 1 - P
    at = y[:, None]
    sure = -torch.expm1(ref["S"].gather(1, at) - ref["lse"][:, None])  # 1 - p without cancellation
    rest.scatter_(1, at, sure)
    dS = P.scatter(1, at, -sure) * dl.double()[:, None]
    small = 2.0 ** -23 * ref["S"].abs().amax(1) + 2.0 ** -21
    u = torch.finfo(dtype).eps / 2
    err = P * (rest * torch.expm1(2 * e)[:, None] + small[:, None]) * dl.double()[:, None]
    err = err + (u + 2.0 ** -22) * (dS.abs() + err) + 2 * 2.0 ** -126
    for name, got, want, a, s, other in (("dX", grads["dX"], dS @ W.double(), dS.abs(), err, Wa),
                                         ("dW", grads["dW"], dS.t() @ X.double(), dS.abs().t(), err.t(), Xa)):
        n = a.shape[1]
        tol = s @ other + (n + 64) * 2.0 ** -23 * (a @ other)
        tol = tol + u * (want.abs() + tol) + 2.0 ** -126
        bad = (got.double() - want).abs() > tol
        assert not bool(bad.any()), (name, int(bad.sum()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,h,V", [(20, 256, 3000), (64, 1024, 2000), (300, 4096, 2000), (600, 8192, 2000), (2500, 2048, 9000)])
def test_confident_tokens(tp, T, h, V, dtype):
    check_confident(tp, T, h, V, dtype)


FEW = [(1, 8, 500), (1, 256, 300), (1, 4096, 9001), (2, 1000, 3000), (3, 4096, 2000), (5, 8192, 1500), (8, 264, 5003)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,h,V", [s for s in FEW if s[1] >= 256])
def test_both_passes_compute_the_same_logits_of_few_tokens(tp, T, h, V, dtype):
    own_bits(tp, T, h, V, dtype)
    own_bits(tp, T, h, V, dtype, piece=136)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,h,V", FEW)
def test_few_confident_tokens(tp, T, h, V, dtype):
    check_confident(tp, T, h, V, dtype)
    check_confident(tp, T, h, V, dtype, piece=64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 2, 4, 6])
def test_gradients_of_few_tokens(tp, T, dtype):
    """Pieces that end inside a group of rows, ignored targets, a target outside the vocabulary, and
    one gradient at a time."""
    h, V = 72, 1003
    for seed in range(4):
        X, W, y, dl = make(T, h, V, dtype, seed=seed, ignored=0.3)
        if seed == 3:
            y[-1] = V
        ctx = tp.XentContext(T, h, V, dtype, piece=(0, 8, 40, 512)[seed])
        loss = tp.xent_forward(ctx, X, W, y)
        assert tp.check_device_status(ctx) == (tp.ERR_INVALID_ARG if seed == 3 else tp.OK)
        grads = tp.xent_backward(ctx, dl)
        assert tp.check_device_status(ctx) == tp.OK
        y = torch.where(y == V, IGN, y)
        check(X, W, y, dl, loss, ctx.lse, grads, reference(X, W, y, dl))
        assert torch.equal(tp.xent_backward(ctx, dl, need_dW=False)["dX"], grads["dX"])
        assert torch.equal(tp.xent_backward(ctx, dl, need_dX=False)["dW"], grads["dW"])


@pytest.mark.parametrize("T,h,V", [(16, 256, 140000), (3, 64, 300000), (40, 4096, 3000), (2100, 1000, 2000),
                                   (700, 8192, 2000), (9000, 512, 700)])
def test_f32_gradients_are_fp32_whatever_the_length(tp, T, h, V):
    """dX and dW as a whole against 64 bits, at K of 700 to 300000.  In units of 2^-24: a product of parts
    is accumulated in ranges of at most 512, 32 steps that cut off a quarter of a unit of the sum on
    average, taken as one and a half times that, 12; the products left out (2^-22) 4; the rounding of dS's
    parts, the sums of ranges and splits 6; in p the logits, at most 3.5, with ranges of 256 (16 steps, 6) and
    four roundings, 35, lse up to 12, 12, and the exponential 8.  They are independent: the root of
    the sum of their squares is 41, and 2^-18 is 64."""
    X, W, y, dl = make(T, h, V, torch.float32, seed=T + h)
    X, W = 0.5 * X, W + 0.01
    ctx, loss, grads = run(tp, X, W, y, dl)
    ref = reference(X, W, y, dl)
    for name in ("dX", "dW"):
        assert float((grads[name].double() - ref[name]).norm()) <= 2.0 ** -18 * float(ref[name].norm()), name


def test_f32_gradients_near_the_ffma_path(tp):
    """The tensor cores' fp32 against the FFMA kernels' on the same inputs: no more than 1.5 times as far
    from 64 bits (both are dominated by sums of about a thousand terms; one accumulation of all of K was
    3 to 9 times as far)."""
    for T, h, V in ((2100, 1000, 2000), (600, 8192, 2000)):
        X, W, y, dl = make(T, h, V, torch.float32, seed=T)
        ref = reference(X, W, y, dl)
        err = {}
        for algo in (tp.ALGO_DEFAULT, tp.ALGO_SIMT):
            _, _, grads = run(tp, X, W, y, dl, algo=algo)
            err[algo] = [float((grads[n].double() - ref[n]).norm() / ref[n].norm()) for n in ("dX", "dW")]
        for a, b in zip(err[tp.ALGO_DEFAULT], err[tp.ALGO_SIMT]):
            assert a <= 1.5 * b, err


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,h,V", [(1, 4096, 3000), (7, 200, 900), (100, 264, 2000), (700, 1000, 9001), (3, 70000, 40)])
def test_scoring_workspace_is_all_the_forward_pass_needs(tp, T, h, V, dtype):
    """The same bits from a workspace of the forward pass's size, and nothing written past it."""
    X, W, y, dl = make(T, h, V, dtype, seed=T)
    for algo in (tp.ALGO_DEFAULT, tp.ALGO_SIMT):
        ctx = tp.XentContext(T, h, V, dtype, algo=algo)
        want = tp.xent_forward(ctx, X, W, y)
        score = tp.XentContext(T, h, V, dtype, algo=algo, backward=False)
        n = score.workspace.numel()
        room = torch.full((n + 65536,), 7, dtype=torch.uint8, device="cuda")
        room[:1024] = 0
        score.workspace = room[:n]
        for _ in range(2):
            assert torch.equal(tp.xent_forward(score, X, W, y), want) and torch.equal(score.lse, ctx.lse)
        assert tp.check_device_status(score) == tp.OK
        assert bool((room[n:] == 7).all())
        with pytest.raises(ValueError):
            tp.xent_backward(score, dl)


@pytest.mark.parametrize("T", [3, 40, 300])
def test_lse_of_the_callers_own(tp, T):
    """It survives the context's next call, and the backward pass reads it."""
    X, W, y, dl = make(T, 128, 900, seed=18)
    X2, _, y2, _ = make(T, 128, 900, seed=19)
    ctx, loss, grads = run(tp, X, W, y, dl)
    want, kept = ctx.lse.clone(), torch.full((T + 2,), 7.0, device="cuda")
    ctx2 = tp.XentContext(T, 128, 900, X.dtype)
    ctx2.lse.fill_(5.0)
    lse = kept[1:T + 1]
    assert torch.equal(tp.xent_forward(ctx2, X, W, y, lse=lse), loss)
    assert bool((ctx2.lse == 5.0).all())
    again = tp.xent_backward(ctx2, dl)
    assert torch.equal(again["dX"], grads["dX"]) and torch.equal(again["dW"], grads["dW"])
    tp.xent_forward(ctx2, X2, W, y2)
    assert torch.equal(lse, want) and float(kept[0]) == 7.0 and float(kept[-1]) == 7.0
    for bad in (torch.empty(T + 1, device="cuda"), torch.empty(T, device="cuda", dtype=torch.bfloat16),
                torch.empty(2 * T, device="cuda")[::2], torch.empty(T)):
        with pytest.raises(ValueError):
            tp.xent_forward(ctx2, X, W, y, lse=bad)


@pytest.mark.parametrize("T,h,V,dtype,piece", [(1, 520, 4000, torch.bfloat16, 0), (6, 520, 4000, torch.bfloat16, 1000),
                                               (3, 130, 4000, torch.float32, 0), (300, 770, 5000, torch.float32, 2048),
                                               (20, 256, 150000, torch.float32, 0), (400, 4096, 3000, torch.bfloat16, 0)])
def test_same_bits_on_every_path(tp, T, h, V, dtype, piece):
    X, W, y, dl = make(T, h, V, dtype, seed=20, ignored=0.1)
    ctx, loss, grads = run(tp, X, W, y, dl, piece=piece)
    lse = ctx.lse.clone()
    for _ in range(3):
        ctx.workspace[1024:] = 255
        assert torch.equal(tp.xent_forward(ctx, X, W, y), loss) and torch.equal(ctx.lse, lse)
        ctx.workspace[1024:] = 255
        again = tp.xent_backward(ctx, dl)
        assert torch.equal(again["dX"], grads["dX"]) and torch.equal(again["dW"], grads["dW"])
