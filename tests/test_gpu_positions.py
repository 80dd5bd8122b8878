"""Norms and rotation of queries and keys, and appending to a paged cache, on the GPU against 64 bits.

Tolerances.  With e = 2^-24 (a rounding of fp32) and u that of the output's type: a component of a rotated pair
(x, y) of normed values is off by u of itself and by K e (|x| + |y|), where K counts the norm (the sum of squares of
16 products and 5 exchanges, halved by the root: 12; the root 2, the products 3), the sine and cosine (2 of their own, 2 for
the angle's 2^-26 of a turn, which is 0.1 e 2^-24 ... 1.6 e) and the rotation (3): 24; 32 is allowed.  Backward, the
same twice over and the mean of dy g xhat: 64, on |r| (|g dy| of the pair + |xhat| mean |g dy xhat|).  The gains'
gradients are sums: e per term added one after the other and per exchange, on the sum of the terms' sizes."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def theta(rot, base=10000.0, scaling=None):
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling is None:
        return f
    if scaling[0] == "linear":
        return [x / scaling[1] for x in f]
    _, factor, context, low, high = scaling
    k = [min(1.0, max(0.0, (context * x / (2 * math.pi) - low) / (high - low))) for x in f]
    return [x * (j + (1 - j) / factor) for x, j in zip(f, k)]


def members(x, rot, layout):
    """u, v of every pair [.., rot/2]."""
    return (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])


def spread(u, v, rest, layout):
    r = torch.cat((u, v), -1) if layout == "half" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((r, rest), -1)


def rotate(x, pos, f, rot, layout, amp=1.0, back=False):
    """The rotation in 64 bits, and the size that its errors go by: |u| + |v| of the pair."""
    if rot == 0:
        return x, x.abs()
    a = pos.double()[:, None, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    c, s = amp * a.cos(), amp * a.sin() * (-1 if back else 1)
    u, v = members(x, rot, layout)
    size = amp * (u.abs() + v.abs()) if amp > 0 else u.abs() + v.abs()
    return (spread(u * c - v * s, u * s + v * c, x[..., rot:], layout),
            spread(size, size, x[..., rot:].abs(), layout))


def split(QKV, heads, kv, d, t):
    n, m = heads // t, kv // t
    x = QKV.view(QKV.shape[0], t, n + 2 * m, d)
    return [x[:, :, a:b].reshape(QKV.shape[0], -1, d) for a, b in ((0, n), (n, n + m), (n + m, n + 2 * m))]


def make(T, heads, kv, d, dt, seed=0, far=1 << 20, norm=True):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    QKV = torch.randn(T, (heads + 2 * kv) * d, generator=g) * torch.exp(0.5 * torch.randn((heads + 2 * kv) * d, generator=g))
    gains = [1 + 0.3 * torch.randn(d, generator=g) for _ in "qk"]
    pos = torch.randint(0, far + 1, (T,), generator=g)
    grads = [torch.randn(T, n, d, generator=g) for n in (heads, kv)]
    return (QKV.to(dt).cuda(), *(x.to(dt).cuda() if norm else None for x in gains), pos.cuda(), *(x.to(dt).cuda() for x in grads))


def forward_reference(x, gain, pos, f, rot, layout, amp):
    x = x.double()
    if gain is not None:
        x = gain.double() * x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    return rotate(x, pos, f, rot, layout, amp)


def check_forward(got, x, gain, pos, f, rot, layout, amp=1.0):
    ref, size = forward_reference(x, gain, pos, f, rot, layout, amp)
    u = torch.finfo(got.dtype).eps / 2
    bad = (got.double() - ref).abs() > u * ref.abs() + 32 * E * size
    assert got.shape == ref.shape and not bool(bad.any()), int(bad.sum())


def backward_reference(x, gain, dy, pos, f, rot, layout, amp=1.0):
    dy, size = rotate(dy.double(), pos, f, rot, layout, amp, back=True)
    if gain is None:
        return dy, size, None, None
    x, g = x.double(), gain.double()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    h = x * r
    m = (dy * g * h).mean(-1, keepdim=True)
    dx = r * (dy * g - h * m)
    dx_size = r * (size * g.abs() + h.abs() * (size * (g * h).abs()).mean(-1, keepdim=True))
    return dx, dx_size, (dy * h).sum((0, 1)), (size * h.abs()).sum((0, 1))


def check_backward(got, dgain, x, gain, dy, pos, f, rot, layout, amp=1.0):
    dx, size, dg, dg_size = backward_reference(x, gain, dy, pos, f, rot, layout, amp)
    u = torch.finfo(got.dtype).eps / 2
    bad = (got.double() - dx).abs() > u * dx.abs() + 64 * E * size
    assert not bool(bad.any()), int(bad.sum())
    if gain is not None:
        n = dy.shape[0] * dy.shape[1]
        bad = (dgain.double() - dg).abs() > u * dg.abs() + (64 + n / 8) * E * dg_size
        assert not bool(bad.any()), int(bad.sum())


CASES = [  # T, heads, kv, d, t, rot, layout, norm
    (1, 1, 1, 2, 1, 2, "half", True), (1, 1, 1, 8, 1, 0, "half", True), (3, 2, 1, 6, 1, 4, "half", True),
    (5, 4, 2, 64, 2, 64, "half", True), (7, 4, 2, 64, 2, 32, "interleaved", True), (33, 3, 3, 80, 1, 48, "half", True),
    (17, 6, 2, 80, 2, 40, "half", True), (17, 6, 2, 80, 2, 40, "interleaved", False), (9, 5, 1, 250, 1, 26, "half", True),
    (65, 8, 8, 96, 4, 96, "interleaved", True), (130, 16, 2, 128, 2, 128, "half", True), (129, 8, 4, 256, 4, 256, "half", False),
    (40, 12, 4, 256, 1, 16, "interleaved", True), (300, 32, 8, 128, 8, 64, "half", True), (2000, 8, 8, 128, 8, 128, "half", True),
    (700, 64, 8, 64, 1, 64, "interleaved", True), (11, 7, 7, 24, 7, 24, "half", True), (4, 2, 2, 36, 1, 34, "half", True),
]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,heads,kv,d,t,rot,layout,norm", CASES)
def test_forward_and_backward_against_64_bits(tp, T, heads, kv, d, t, rot, layout, norm, dt):
    QKV, gq, gk, pos, dQ, dK = make(T, heads, kv, d, dt, T + d, norm=norm)
    rope = tp.RopeTable(rot, layout=layout) if rot else None
    ctx = tp.QkContext(T, heads, kv, d, dt, rope, norm=norm, eps=EPS, t=t)
    before = QKV.clone()
    Qr, Kr = tp.qk_forward(ctx, QKV, pos, gq, gk)
    Q, K, V = split(QKV, heads, kv, d, t)
    f = theta(rot) if rot else []
    check_forward(Qr, Q, gq, pos, f, rot, layout)
    check_forward(Kr, K, gk, pos, f, rot, layout)
    g = tp.qk_backward(ctx, dQ, dK)
    check_backward(g["dQ"], g["dgain_q"], Q, gq, dQ, pos, f, rot, layout)
    check_backward(g["dK"], g["dgain_k"], K, gk, dK, pos, f, rot, layout)
    assert torch.equal(QKV, before) and tp.check_device_status(ctx) == tp.OK
    # the same bits from arrays laid out as QKV, into one whose V columns stay
    out = torch.full_like(QKV, 7.0)
    assert tp.qk_forward(ctx, QKV, pos, gq, gk, out=out) is out
    o = split(out, heads, kv, d, t)
    assert torch.equal(o[0], Qr) and torch.equal(o[1], Kr) and bool((o[2] == 7).all())
    out = torch.full_like(QKV, 7.0)
    g2 = tp.qk_backward(ctx, dQ, dK, out=out)
    o = split(g2["dQKV"], heads, kv, d, t)
    assert torch.equal(o[0], g["dQ"]) and torch.equal(o[1], g["dK"]) and bool((o[2] == 7).all())
    if norm:
        assert torch.equal(g2["dgain_q"], g["dgain_q"]) and torch.equal(g2["dgain_k"], g["dgain_k"])


@pytest.mark.parametrize("scaling", [("linear", 4.0), ("parts", 8.0, 2048, 1.0, 32.0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions_and_scaling(tp, scaling, layout):
    T, heads, kv, d = 64, 2, 1, 128
    QKV, _, _, _, dQ, dK = make(T, heads, kv, d, torch.float32, 5, norm=False)
    pos = torch.tensor([0, 1, 2, 3, -1, -5, 1 << 20, (1 << 24) + 1, (1 << 31) + 7] * 8)[:T].cuda()
    ctx = tp.QkContext(T, heads, kv, d, torch.float32, tp.RopeTable(d, 500000.0, layout, scaling, 1.25), norm=False)
    Qr, Kr = tp.qk_forward(ctx, QKV, pos)
    Q, K, _ = split(QKV, heads, kv, d, 1)
    f = theta(d, 500000.0, scaling)
    # position * theta in 64 bits is itself off by 2^-53 of it, under 2^-22 turns at 2^31: compared there to 2^-20
    near = pos.abs() < 1 << 25
    check_forward(Qr[near], Q[near], None, pos[near], f, d, layout, 1.25)
    ref, size = rotate(Q[~near].double(), pos[~near], f, d, layout, 1.25)
    assert bool(((Qr[~near].double() - ref).abs() <= 2.0 ** -20 * size + 32 * E * size).all())
    g = tp.qk_backward(ctx, dQ, dK)
    check_backward(g["dQ"][near], None, Q[near], None, dQ[near], pos[near], f, d, layout, 1.25)
    assert g["dgain_q"] is None


def test_formula_against_differences():
    """The gradients that the kernels are compared with, against differences of the forward formula in 64 bits."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 2, 16, generator=g, dtype=torch.float64)
    gain, w = 1 + torch.randn(16, generator=g, dtype=torch.float64), torch.randn(3, 2, 16, generator=g, dtype=torch.float64)
    pos, f = torch.tensor([0, 5, 900]), theta(12)

    def loss(x, gain):
        return float((forward_reference(x, gain, pos, f, 12, "half", 1.5)[0] * w).sum())

    dx, _, dg, _ = backward_reference(x, gain, w, pos, f, 12, "half", 1.5)
    step = 1e-5
    for i in range(0, 96, 7):
        h = torch.zeros(96, dtype=torch.float64)
        h[i] = step
        h = h.view_as(x)
        assert abs((loss(x + h, gain) - loss(x - h, gain)) / (2 * step) - float(dx.flatten()[i])) < 1e-7
    for i in range(16):
        h = torch.zeros(16, dtype=torch.float64)
        h[i] = step
        assert abs((loss(x, gain + h) - loss(x, gain - h)) / (2 * step) - float(dg[i])) < 1e-7


def test_strided_rows_in_place_and_guards(tp):
    T, heads, kv, d, dt = 50, 4, 2, 64, torch.bfloat16
    QKV, gq, gk, pos, dQ, dK = make(T, heads, kv, d, dt, 9)
    wide = torch.full((T, QKV.shape[1] + 24), 3.0, dtype=dt, device="cuda")
    wide[:, 8:-16] = QKV
    view = wide[:, 8:-16]
    ctx = tp.QkContext(T, heads, kv, d, dt, tp.RopeTable(d), eps=EPS)
    Qr, Kr = tp.qk_forward(ctx, QKV, pos, gq, gk)
    a, b = tp.qk_forward(ctx, view, pos, gq, gk)
    assert torch.equal(a, Qr) and torch.equal(b, Kr)
    odd = torch.full((T, QKV.shape[1] + 3), 3.0, dtype=dt, device="cuda")[:, 1:-2]  # rows on two bytes
    odd.copy_(QKV)
    a, b = tp.qk_forward(ctx, odd, pos, gq, gk)
    f = theta(d)
    for got, x, gain in zip((a, b), split(QKV, heads, kv, d, 1), (gq, gk)):
        check_forward(got, x, gain, pos, f, d, "half")
    # in place: the same values, V and the columns around untouched, and no backward pass from it
    assert tp.qk_forward(ctx, view, pos, gq, gk, out=view) is view
    o = split(view.contiguous(), heads, kv, d, 1)
    assert torch.equal(o[0], Qr) and torch.equal(o[1], Kr) and torch.equal(o[2], split(QKV, heads, kv, d, 1)[2])
    assert bool((wide[:, :8] == 3).all()) and bool((wide[:, -16:] == 3).all())
    with pytest.raises(ValueError):
        tp.qk_backward(ctx, dQ, dK)
    # separate tensors
    Q, K, V = split(QKV, heads, kv, d, 1)
    a, b = tp.qk_forward(ctx, (Q, K), pos, gq, gk)
    assert torch.equal(a, Qr) and torch.equal(b, Kr)
    # gradients in place
    want = tp.qk_backward(ctx, dQ, dK)
    g = tp.qk_backward(ctx, dQ, dK, out=(dQ, dK))
    assert g["dQ"] is dQ and torch.equal(dQ, want["dQ"]) and torch.equal(dK, want["dK"])


def test_no_tokens(tp):
    ctx = tp.QkContext(0, 4, 2, 64, torch.float32, tp.RopeTable(64))
    one = torch.ones(64, device="cuda")
    Q, K = tp.qk_forward(ctx, torch.empty(0, 512, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), one, one)
    g = tp.qk_backward(ctx, Q, K)
    assert bool((g["dgain_q"] == 0).all()) and bool((g["dgain_k"] == 0).all()) and Q.shape == (0, 4, 64)


def test_zero_and_non_finite_rows_stay_alone(tp):
    T, heads, kv, d = 8, 2, 2, 64
    QKV, gq, gk, pos, dQ, dK = make(T, heads, kv, d, torch.float32, 11)
    QKV[2, :d] = 0.0
    clean = QKV.clone()
    QKV[4, 0] = float("nan")
    QKV[5, d] = float("inf")
    ctx = tp.QkContext(T, heads, kv, d, torch.float32, tp.RopeTable(d), eps=EPS)
    Qr, Kr = tp.qk_forward(ctx, QKV, pos, gq, gk)
    Qc, Kc = tp.qk_forward(ctx, clean, pos, gq, gk)
    assert bool((Qr[2, 0] == 0).all()) and torch.equal(Kr, Kc)
    same = torch.ones(T, heads, dtype=torch.bool, device="cuda")
    same[4, 0] = same[5, 1] = False
    assert torch.equal(Qr[same], Qc[same]) and not bool(Qr[4, 0].isfinite().any())


def test_other_streams_and_replays(tp):
    T, heads, kv, d, dt = 256, 8, 2, 128, torch.bfloat16
    QKV, gq, gk, pos, dQ, dK = make(T, heads, kv, d, dt, 1)
    ctx = tp.QkContext(T, heads, kv, d, dt, tp.RopeTable(d))
    want = tp.qk_forward(ctx, QKV, pos, gq, gk)
    grads = tp.qk_backward(ctx, dQ, dK)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = tp.qk_forward(ctx, QKV, pos, gq, gk)
        got2 = tp.qk_backward(ctx, dQ, dK)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(got2[k], grads[k]) for k in grads)
    x, p = QKV.clone(), pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tp.qk_forward(ctx, x, p, gq, gk)
        back = tp.qk_backward(ctx, dQ, dK)
    x.copy_(QKV.flip(0))
    p.copy_(pos.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0].flip(0)) and torch.equal(out[1], want[1].flip(0))
    assert back["dQ"].isfinite().all()


# ---- append ------------------------------------------------------------------------------------

APPEND = [  # T, heads, kv, d, t, rot, layout, norm, page, dtype
    (1, 4, 4, 64, 1, 64, "half", True, 16, torch.bfloat16), (1, 32, 8, 128, 8, 128, "half", True, 16, torch.bfloat16),
    (37, 6, 2, 80, 2, 32, "interleaved", True, 7, torch.bfloat16), (100, 4, 1, 24, 1, 10, "half", False, 1, torch.float32),
    (300, 16, 2, 256, 1, 256, "half", True, 48, torch.bfloat16), (2050, 8, 8, 128, 1, 64, "interleaved", True, 64, torch.bfloat16),
    (63, 3, 3, 8, 1, 8, "half", True, 5, torch.float32), (20, 2, 2, 64, 1, 0, "half", True, 16, torch.float32),
]


def cache_of(tp, pages, kv, page, d, dt, order, seed=0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    if order == "tokens":
        K, V = (torch.randn(pages, page, kv, d, generator=g).to(dt).cuda().transpose(1, 2) for _ in "kv")
    elif order == "together":  # K and V of a page one after the other
        both = torch.randn(pages, 2, kv, page, d, generator=g).to(dt).cuda()
        K, V = both[:, 0], both[:, 1]
    else:
        K, V = (torch.randn(pages, kv, page, d, generator=g).to(dt).cuda() for _ in "kv")
    return tp.KvCache.of(K, V)


@pytest.mark.parametrize("order", ["heads", "tokens", "together"])
@pytest.mark.parametrize("T,heads,kv,d,t,rot,layout,norm,page,dt", APPEND)
def test_append(tp, T, heads, kv, d, t, rot, layout, norm, page, dt, order):
    QKV, gq, gk, pos, _, _ = make(T, heads, kv, d, dt, T, norm=norm)
    pages = (T + page - 1) // page + 3
    cache = cache_of(tp, pages, kv, page, d, dt, order)
    slot = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:T].cuda()
    slot[2::5] = -1
    K0, V0 = cache.K.clone(), cache.V.clone()
    rope = tp.RopeTable(rot, layout=layout) if rot else None
    ctx = tp.QkContext(T, heads, kv, d, dt, rope, norm=norm, eps=EPS, t=t)
    Qr = tp.kv_append(ctx, cache, QKV, pos, slot, gq, gk)
    assert tp.check_device_status(ctx) == tp.OK
    # the same bits as the rotation alone, in the rows of the slots and nowhere else
    Q, K = tp.qk_forward(ctx, QKV, pos, gq, gk)
    V = split(QKV, heads, kv, d, t)[2]
    kept = slot >= 0
    at = slot[kept]
    K0[at // page, :, at % page] = K[kept]
    V0[at // page, :, at % page] = V[kept]
    assert torch.equal(Qr, Q) and torch.equal(cache.K, K0) and torch.equal(cache.V, V0)
    # into the queries' own columns
    out = split(QKV, heads, kv, d, t)[0] if t == 1 else None
    if t == 1:
        inside = QKV[:, :heads * d].view(T, heads, d)
        assert tp.kv_append(ctx, cache, QKV, pos, slot, gq, gk, out=inside) is inside
        assert torch.equal(inside, Q) and torch.equal(cache.K, K0) and out is not None


def test_a_slot_outside_the_cache_is_reported(tp):
    T, heads, kv, d, dt = 6, 2, 2, 64, torch.bfloat16
    QKV, gq, gk, pos, _, _ = make(T, heads, kv, d, dt, 2)
    cache = cache_of(tp, 3, kv, 4, d, dt, "heads")
    K0 = cache.K.clone()
    ctx = tp.QkContext(T, heads, kv, d, dt, tp.RopeTable(d))
    slot = torch.tensor([0, 12, -7, 5, 1 << 40, -(1 << 62)], device="cuda")
    Qr = tp.kv_append(ctx, cache, QKV, pos, slot, gq, gk)
    assert int(ctx.workspace[4:8].view(torch.int32)[0]) in (1, 4)
    assert tp.check_device_status(ctx) == tp.ERR_INVALID_ARG
    Q, K = tp.qk_forward(ctx, QKV, pos, gq, gk)
    K0[0, :, 0], K0[1, :, 1] = K[0], K[3]
    assert torch.equal(Qr, Q) and torch.equal(cache.K, K0)
    assert tp.check_device_status(ctx) == tp.OK


def test_a_cache_past_32_bits(tp):
    T, heads, kv, d, dt = 5, 2, 2, 128, torch.bfloat16
    pages, page = 1 << 15, 300  # 2.5 G elements each
    QKV, gq, gk, pos, _, _ = make(T, heads, kv, d, dt, 4)
    K, V = (torch.empty(pages, kv, page, d, dtype=dt, device="cuda") for _ in "kv")
    cache = tp.KvCache.of(K, V)
    slot = torch.tensor([0, pages * page - 1, (pages - 2) * page + 7, pages // 2 * page, -1], device="cuda")
    ctx = tp.QkContext(T, heads, kv, d, dt, tp.RopeTable(d))
    tp.kv_append(ctx, cache, QKV, pos, slot, gq, gk)
    _, Kr = tp.qk_forward(ctx, QKV, pos, gq, gk)
    for i in range(4):
        p, r = divmod(int(slot[i]), page)
        assert torch.equal(K[p, :, r], Kr[i]) and torch.equal(V[p, :, r], split(QKV, heads, kv, d, 1)[2][i])
