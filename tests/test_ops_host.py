"""Host side of the vocabulary cross entropy and the orthogonalisation, without a GPU: sizes,
argument checks that fail before any CUDA call (no pointer is ever dereferenced), and
the index arithmetic of the symmetric tiles, the transposed staging box and the operand parts,
restated."""
import ctypes

import pytest

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import build
    build.build()
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def xshape(tp, T=64, h=256, V=1000, ignore=-100, piece=0, dtype=None, algo=0):
    return tp.XentShape(T, h, V, ignore, piece, tp.BF16 if dtype is None else dtype, algo)


def xws(tp, s):
    return tp.lib.tpmlp_xent_workspace_bytes(ctypes.byref(s))


def test_xent_workspace(tp):
    assert xws(tp, xshape(tp)) > 0
    assert xws(tp, xshape(tp, T=0)) > 0
    for bad in (dict(T=-1), dict(h=0), dict(V=0), dict(piece=-8), dict(piece=12), dict(dtype=7), dict(algo=5),
                dict(T=1 << 30, V=1 << 30)):
        assert xws(tp, xshape(tp, **bad)) == 0, bad
    # the logits are not kept: 8192 tokens and 65536 vocabulary rows are 1 GiB in bf16
    assert xws(tp, xshape(tp, T=8192, h=4096, V=65536)) < 600 << 20
    # a smaller piece needs less
    assert xws(tp, xshape(tp, T=8192, h=4096, V=65536, piece=4096)) < xws(tp, xshape(tp, T=8192, h=4096, V=65536))


def xfwd(tp, s, p=None, ws=FAKE):
    p = p or [FAKE] * 5
    return tp.lib.tpmlp_xent_forward(ctypes.byref(s) if s is not None else None, *p, ws, None)


def xbwd(tp, s, p=None, ws=FAKE):
    p = p or [FAKE] * 7
    return tp.lib.tpmlp_xent_backward(ctypes.byref(s) if s is not None else None, *p, ws, None)


def test_xent_refusals(tp):
    good = xshape(tp)
    assert xfwd(tp, None) == tp.ERR_INVALID_ARG and xbwd(tp, None) == tp.ERR_INVALID_ARG
    assert xfwd(tp, xshape(tp, V=0)) == tp.ERR_INVALID_ARG
    assert xfwd(tp, good, ws=None) == tp.ERR_INVALID_ARG and xbwd(tp, good, ws=None) == tp.ERR_INVALID_ARG
    for i in range(5):
        assert xfwd(tp, good, [None if k == i else FAKE for k in range(5)]) == tp.ERR_INVALID_ARG
    for i in range(5):  # dX and dW (5, 6) may be NULL
        assert xbwd(tp, good, [None if k == i else FAKE for k in range(7)]) == tp.ERR_INVALID_ARG
    assert xbwd(tp, good, [FAKE] * 5 + [None, None]) == tp.OK  # nothing asked for
    apart = [FAKE + 4096 * k for k in range(7)]
    for i, j in ((5, 0), (5, 1), (6, 0), (6, 1), (6, 5)):  # outputs in the place of inputs, or of each other
        assert xbwd(tp, good, [apart[j] if k == i else apart[k] for k in range(7)]) == tp.ERR_INVALID_ARG
    for i in (0, 1):  # X and W on 16 bytes
        assert xfwd(tp, good, [FAKE + 2 if k == i else FAKE for k in range(5)]) == tp.ERR_UNSUPPORTED
        assert "16-byte" in tp.last_error()
    for i in (5, 6):
        assert xbwd(tp, good, [apart[k] + (2 if k == i else 0) for k in range(7)]) == tp.ERR_UNSUPPORTED
    assert xfwd(tp, good, [FAKE, FAKE, FAKE + 4, FAKE, FAKE]) == tp.ERR_UNSUPPORTED  # int64 targets
    assert xfwd(tp, xshape(tp, h=250)) == tp.ERR_UNSUPPORTED
    assert xfwd(tp, xshape(tp, T=65535 * 64 + 1, h=8, V=8, algo=1)) == tp.ERR_UNSUPPORTED
    # no tokens: the token arrays may be NULL
    assert xfwd(tp, xshape(tp, T=0), [None, FAKE, None, None, None]) == tp.OK


def test_xent_outputs_overlap_nothing(tp):
    """T = 64, h = 256, V = 1000 in bf16: X 32768 bytes, W 512000, targets 512, fp32 rows 256.  An
    output one byte range into any other buffer is refused, from below and from above."""
    good = xshape(tp)
    size = {"X": 32768, "W": 512000, "target": 512, "loss": 256, "lse": 256, "dloss": 256, "dX": 32768, "dW": 512000}
    at = {n: (k + 1) << 20 for k, n in enumerate(size)}
    for call, names, outs in ((xfwd, ("X", "W", "target", "loss", "lse"), ("loss", "lse")),
                              (xbwd, ("X", "W", "target", "lse", "dloss", "dX", "dW"), ("dX", "dW"))):
        for out in outs:
            for other in names:
                if other == out:
                    continue
                for where in (at[other] + size[other] - 16, at[other] - size[out] + 16):
                    p = [where if n == out else at[n] for n in names]
                    assert call(tp, good, p) == tp.ERR_INVALID_ARG, (out, other)
                    assert "overlaps" in tp.last_error()


def oshape(tp, batch=2, rows=64, cols=128, steps=5, dtype=None, coef=(3.4445, -4.7750, 2.0315), eps=1e-7):
    return tp.OrthoShape(batch, rows, cols, steps, tp.BF16 if dtype is None else dtype, *coef, eps)


def test_ortho_workspace_and_refusals(tp):
    ws = lambda s: tp.lib.tpmlp_ortho_workspace_bytes(ctypes.byref(s))
    assert ws(oshape(tp)) > 0 and ws(oshape(tp, batch=0)) > 0
    inf, nan = float("inf"), float("nan")
    for bad in (dict(batch=-1), dict(batch=65536), dict(rows=0), dict(cols=0), dict(rows=(1 << 20) + 1), dict(steps=0),
                dict(steps=33), dict(dtype=9), dict(eps=-1.0), dict(eps=inf), dict(eps=nan),
                dict(rows=1 << 20, cols=1 << 20)):
        assert ws(oshape(tp, **bad)) == 0, bad
    call = lambda s, G=FAKE, O=FAKE, w=FAKE: tp.lib.tpmlp_orthogonalize(ctypes.byref(s), G, O, w, None)
    assert tp.lib.tpmlp_orthogonalize(None, FAKE, FAKE, FAKE, None) == tp.ERR_INVALID_ARG
    assert call(oshape(tp), G=None) == tp.ERR_INVALID_ARG
    assert call(oshape(tp), O=None) == tp.ERR_INVALID_ARG
    assert call(oshape(tp), w=None) == tp.ERR_INVALID_ARG
    assert call(oshape(tp), w=FAKE + 8) == tp.ERR_UNSUPPORTED
    assert call(oshape(tp), O=FAKE + 2) == tp.ERR_UNSUPPORTED       # rows of 16 bytes want the base there too
    assert call(oshape(tp, cols=127), O=FAKE + 1) == tp.ERR_UNSUPPORTED
    assert call(oshape(tp, dtype=tp.F32), G=FAKE + 2) == tp.ERR_UNSUPPORTED
    # iterates that grow: 2 s at every step; a polynomial that is not one
    for coef in ((2.0, 0.0, 0.0), (30.0, -4.0, 2.0), (nan, 0.0, 0.0), (3.4445, -4.775, inf), (-9.0, 0.0, 0.0)):
        assert call(oshape(tp, coef=coef)) == tp.ERR_UNSUPPORTED, coef
        assert "fp16" in tp.last_error()
    assert call(oshape(tp, batch=0), G=None, O=None) == tp.OK


def test_symmetric_tiles_cover_the_lower_triangle_once():
    """Tile i of a symmetric product of n x n tiles: the root of 8 i + 1 in fp32, put right by
    the two loops, gives row mb and column nb <= mb."""
    import numpy as np
    for n in (1, 2, 3, 16, 100, 400):
        seen = set()
        for i in range(n * (n + 1) // 2):
            mb = int((np.sqrt(np.float32(8.0) * np.float32(i) + np.float32(1.0)) - np.float32(1.0)) * np.float32(0.5))
            while mb * (mb + 1) // 2 > i:
                mb -= 1
            while (mb + 1) * (mb + 2) // 2 <= i:
                mb += 1
            nb = i - mb * (mb + 1) // 2
            assert 0 <= nb <= mb < n
            seen.add((mb, nb))
        assert len(seen) == n * (n + 1) // 2


def test_transposed_box():
    """The exchange with the neighbouring lane and the swizzled store of a 32 x 32 box of 16-bit
    values, against the transpose; every store of the 32 lanes touches 32 different banks."""
    box = [[100 * r + c for c in range(32)] for r in range(32)]
    words = [[(box[r][2 * i], box[r][2 * i + 1]) for i in range(16)] for r in range(32)]
    smem = {}
    for i in range(16):
        banks = set()
        for lane in range(32):
            odd, other, mine = lane & 1, words[lane ^ 1][i], words[lane][i]
            t = (other[1], mine[1]) if odd else (mine[0], other[0])
            r, word = 2 * i + odd, lane >> 1
            at = r * 64 + (((word >> 2) ^ ((r >> 1) & 3)) << 4) + ((word & 3) << 2)
            banks.add(at // 4 % 32)
            assert at not in smem
            smem[at] = t
        assert len(banks) == 32
    for r in range(32):  # read back as a 64-byte-swizzled box
        for c in range(32):
            chunk = (c * 2 >> 4) ^ ((r >> 1) & 3)
            at = r * 64 + (chunk << 4) + (c * 2 & 12)
            assert smem[at][c & 1] == box[c][r]


def test_three_parts_hold_a_float():
    """Each part the rest rounded to bf16: the three add up to the fp32 number exactly, and the six
    products that are taken leave out at most 2 * 2^-8 * 2^-16 + 2^-32 < 2^-22 of |a| |b| (a part
    is at most 2^-8 of the one before it: half a step of an eight-bit significand)."""
    import numpy as np

    def bf16(x):
        u = x.view(np.uint32)
        u = u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))
        return (u & np.uint32(0xFFFF0000)).view(np.float32)

    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * np.exp2(rng.integers(-60, 60, 20000))).astype(np.float32)
    p0 = bf16(x)
    p1 = bf16(x - p0)
    p2 = x - p0 - p1
    assert np.array_equal(p2, bf16(p2))  # eight bits are left: a bf16 number
    assert np.array_equal(p0.astype(np.float64) + p1 + p2, x.astype(np.float64))
    a, b = (x[:10000], x[10000:])
    pa = [v[:10000].astype(np.float64) for v in (p0, p1, p2)]
    pb = [v[10000:].astype(np.float64) for v in (p0, p1, p2)]
    seg_a, seg_b = (0, 2, 1, 0, 1, 0), (2, 0, 1, 1, 0, 0)
    got = sum(pa[i] * pb[j] for i, j in zip(seg_a, seg_b))
    exact = a.astype(np.float64) * b
    assert np.all(np.abs(got - exact) <= 2.0 ** -22 * np.abs(exact))


def test_bindings(tp):
    import torch
    with pytest.raises(ValueError):
        tp.XentContext(4, 8, 0, torch.bfloat16, device="cpu")
    with pytest.raises(ValueError):
        tp.XentContext(4, 8, 16, torch.float16, device="cpu")
    with pytest.raises(ValueError):
        tp.OrthoContext(0, 8, device="cpu")
    with pytest.raises(ValueError):
        tp.OrthoContext(8, 8, dtype=torch.float16, device="cpu")
    ctx = tp.XentContext(4, 8, 16, torch.float32, device="cpu")  # buffers only; calls refuse CPU tensors
    with pytest.raises(ValueError):
        tp.xent_forward(ctx, torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(4, dtype=torch.int64))


def test_no_tokens_at_any_hidden_size(tp):
    """T = 0 is a valid shape whatever the hidden size: also past the 98304 (bf16), 49152 (fp32) and 12256
    (bf16, more than one token) elements up to which X fits the few-token kernels' shared memory."""
    for dtype in (tp.BF16, tp.F32):
        for algo in (0, 1):
            for h in (8, 12256, 12264, 49152, 49160, 98304, 98312, 1 << 20):
                s = xshape(tp, T=0, h=h, V=100, dtype=dtype, algo=algo)
                assert xws(tp, s) > 0
                assert xfwd(tp, s, [None, FAKE, None, None, None]) == tp.OK
                assert xbwd(tp, s, [None, FAKE, None, None, None, None, None]) == tp.OK


def test_scoring_workspace(tp):
    """The forward pass alone: no dS, no sums of dX and dW, and for few tokens no parts of W."""
    fwd = lambda **k: tp.lib.tpmlp_xent_forward_workspace_bytes(ctypes.byref(xshape(tp, **k)))
    for k in (dict(), dict(T=1, h=4096, V=32768), dict(T=4, h=4096, V=128256, dtype=tp.F32), dict(T=0),
              dict(T=300, h=770, V=2500, dtype=tp.F32), dict(algo=1), dict(algo=1, dtype=tp.F32), dict(piece=64)):
        assert 0 < fwd(**k) <= xws(tp, xshape(tp, **k)), k
    for bad in (dict(T=-1), dict(h=0), dict(V=0), dict(piece=12), dict(dtype=7), dict(algo=5)):
        assert fwd(**bad) == 0, bad
    assert fwd(T=4, h=4096, V=128256, dtype=tp.F32) < 1 << 20
    # two (max, sum) pairs of 8 bytes per token and at most 256 vocabulary rows
    assert fwd(T=8192, h=4096, V=65536) <= 8192 * (65536 // 256) * 16 + (1 << 20)
    # fp32 in three parts of 2 bytes
    assert fwd(T=100, h=256, V=1000, dtype=tp.F32) >= 6 * 256 * 1100


def test_scoring_context_refuses_the_backward_pass(tp):
    import torch
    ctx = tp.XentContext(4, 4096, 128256, torch.float32, device="cpu", backward=False)
    assert ctx.workspace.numel() < 1 << 20
    ctx._saved = (None, None, None)
    with pytest.raises(ValueError, match="backward=False"):
        tp.xent_backward(ctx, torch.zeros(4))
