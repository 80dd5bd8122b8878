"""ctypes binding of libtpmlp.so (C ABI in include/tpmlp.h): argument marshalling
only.  Every step of the forward and backward pass runs in the library's CUDA
kernels; PyTorch supplies device memory and the current stream.

Importing this module loads the compiled library and raises if it is missing:
there is no fallback implementation.  TPMLP_LIBRARY=debug (read at import)
loads libtpmlp_debug.so instead, the build whose GEMM kernels bounds-check every
tile access and report a failed check as ERR_DEVICE in the status word.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtpmlp_debug.so" if os.environ.get("TPMLP_LIBRARY") == "debug"
                        else "libtpmlp.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_DEVICE = range(6)
F32, BF16 = 0, 1
ALGO_DEFAULT, ALGO_SIMT = 0, 1
WS_STATUS, WS_PARTIALS, WS_DY, WS_Y, WS_DXN = 0, 1, 2, 3, 4
FLAG_RECOMPUTE, FLAG_LAYERNORM = 1, 2
ATTN_P_UPPER_ZERO = 1
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_PARTS = 0, 1, 2

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


class Shape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("ffn", ctypes.c_int64),
                ("t", ctypes.c_int32), ("dtype", ctypes.c_int32), ("algo", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class Saved(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("H", ctypes.c_void_p), ("Y", ctypes.c_void_p)]


class LayerNorm(ctypes.Structure):
    _fields_ = [("X_in", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("Xn", ctypes.c_void_p), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class AttnShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seq", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("t", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class AttnSaved(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("Wqkv", ctypes.c_void_p), ("Wo", ctypes.c_void_p),
                ("QKV", ctypes.c_void_p), ("P", ctypes.c_void_p), ("O", ctypes.c_void_p)]


class XentShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("ignore_index", ctypes.c_int64), ("piece", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("algo", ctypes.c_int32)]


class OrthoShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("steps", ctypes.c_int32), ("dtype", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("eps", ctypes.c_float)]


class Rope(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("context", ctypes.c_int64), ("rot", ctypes.c_int32),
                ("scaling", ctypes.c_int32)]


class QkShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("t", ctypes.c_int32), ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("rot", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("amplitude", ctypes.c_float)]


class Heads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("row", ctypes.c_int64), ("shard", ctypes.c_int64)]


class KvCacheShape(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class CacheAttnShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("batch", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("tree_words", ctypes.c_int32), ("algo", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class TpmlpError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = last_error()
        super().__init__("%s: %s (status %d)%s" % (what, status_string(status), status,
                                                    (": " + detail) if detail else ""))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("%s is not built (expected at %s); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`"
                          % (os.path.basename(LIB_PATH), LIB_PATH))
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, i64, u64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64
    SP = ctypes.POINTER(Shape)
    decl = {
        "tpmlp_status_string": (ctypes.c_char_p, [i32]),
        "tpmlp_version": (i32, []),
        "tpmlp_last_error": (ctypes.c_char_p, []),
        "tpmlp_saved_bytes": (sz, [SP]),
        "tpmlp_workspace_bytes": (sz, [SP]),
        "tpmlp_workspace_offset": (sz, [SP, i32]),
        "tpmlp_forward": (i32, [SP, vp, vp, vp, vp, vp, vp, ctypes.POINTER(Saved), vp, vp]),
        "tpmlp_backward": (i32, [SP, vp, ctypes.POINTER(Saved), vp, vp, vp, vp, vp, vp, vp]),
        "tpmlp_ln_forward": (i32, [SP, ctypes.POINTER(LayerNorm), vp]),
        "tpmlp_ln_backward": (i32, [SP, ctypes.POINTER(LayerNorm), vp, vp, vp, vp, vp, vp]),
        "tpmlp_sp_forward": (i32, [SP, ctypes.POINTER(LayerNorm), vp, vp, vp, vp, vp, ctypes.POINTER(Saved),
                                   vp, vp]),
        "tpmlp_sp_backward": (i32, [SP, ctypes.POINTER(LayerNorm), vp, ctypes.POINTER(Saved)] + [vp] * 9),
        "tpmlp_attn_saved_bytes": (sz, [ctypes.POINTER(AttnShape)]),
        "tpmlp_attn_workspace_bytes": (sz, [ctypes.POINTER(AttnShape)]),
        "tpmlp_attn_forward": (i32, [ctypes.POINTER(AttnShape)] + [vp] * 6 + [ctypes.POINTER(AttnSaved), vp, vp]),
        "tpmlp_attn_backward": (i32, [ctypes.POINTER(AttnShape), vp, ctypes.POINTER(AttnSaved)] + [vp] * 7),
        "tpmlp_xent_workspace_bytes": (sz, [ctypes.POINTER(XentShape)]),
        "tpmlp_xent_forward_workspace_bytes": (sz, [ctypes.POINTER(XentShape)]),
        "tpmlp_xent_forward": (i32, [ctypes.POINTER(XentShape)] + [vp] * 7),
        "tpmlp_xent_backward": (i32, [ctypes.POINTER(XentShape)] + [vp] * 9),
        "tpmlp_ortho_workspace_bytes": (sz, [ctypes.POINTER(OrthoShape)]),
        "tpmlp_orthogonalize": (i32, [ctypes.POINTER(OrthoShape)] + [vp] * 4),
        "tpmlp_rope_turns": (i32, [ctypes.POINTER(Rope), vp]),
        "tpmlp_qk_workspace_bytes": (sz, [vp]),
        "tpmlp_qk_forward": (i32, [vp] * 10),
        "tpmlp_qk_backward": (i32, [vp] * 15),
        "tpmlp_kv_append": (i32, [vp] * 13),
        "tpmlp_cache_attn_workspace_bytes": (sz, [vp, vp]),
        "tpmlp_cache_attn": (i32, [vp] * 10),
        "tpmlp_check_device_status": (i32, [vp, vp]),
        "tpmlp_set_wait_limit_ns": (None, [u64]),
        "tpmlp_debug_timeout_probe": (i32, [vp, u64, vp]),
        "tpmlp_launch_count": (u64, []),
        "tpmlp_profile_enable": (None, [i32]),
        "tpmlp_profile_reset": (None, []),
        "tpmlp_profile_collect": (i32, []),
        "tpmlp_profile_count": (i32, []),
        "tpmlp_profile_entry": (i32, [i32, ctypes.c_char_p, i32, ctypes.POINTER(i64),
                                      ctypes.POINTER(ctypes.c_double)]),
    }
    for name, (res, args) in decl.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.tpmlp_status_string(int(status)).decode()


def last_error() -> str:
    return lib.tpmlp_last_error().decode(errors="replace")


def make_shape(tokens: int, hidden: int, ffn: int, t: int, dtype, algo: int = ALGO_DEFAULT,
               flags: int = 0) -> Shape:
    if isinstance(dtype, torch.dtype):
        dtype = _DTYPES[dtype]
    return Shape(int(tokens), int(hidden), int(ffn), int(t), int(dtype), int(algo), int(flags))


def saved_bytes(shape: Shape) -> int:
    return int(lib.tpmlp_saved_bytes(ctypes.byref(shape)))


def workspace_bytes(shape: Shape) -> int:
    return int(lib.tpmlp_workspace_bytes(ctypes.byref(shape)))


def workspace_offset(shape: Shape, region: int) -> int:
    return int(lib.tpmlp_workspace_offset(ctypes.byref(shape), int(region)))


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(status: int, what: str):
    if status != OK:
        raise TpmlpError(status, what)


def _need(x, name, dtype, shape):
    if x.is_cuda and x.dtype is dtype and x.shape == shape and x.is_contiguous():
        return
    if not (x.is_cuda and x.is_contiguous()):
        raise ValueError("%s must be a contiguous CUDA tensor" % name)
    if x.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, x.dtype, dtype))
    if tuple(x.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(x.shape), tuple(shape)))


def new_workspace(shape: Shape, device=None) -> torch.Tensor:
    """A zeroed workspace of the size the library asks for (uint8, 256-byte aligned)."""
    n = workspace_bytes(shape)
    if n == 0:
        raise ValueError("invalid shape")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


class Context:
    """The buffers one layer needs between forward and backward: H, Y and the
    workspace, plus the ctypes shape and saved-activation records."""

    def __init__(self, tokens, hidden, ffn, t, dtype, algo=ALGO_DEFAULT, device=None, keep_H=True,
                 recompute=False, layernorm=False, eps=1e-5):
        """recompute=True keeps only H between the passes (TPMLP_FLAG_RECOMPUTE):
        Y then lives in the workspace and is rebuilt by the backward pass.
        layernorm=True adds the LayerNorm in front (the sequence-parallel block,
        TPMLP_FLAG_LAYERNORM): Xn, mean and rstd buffers are allocated here."""
        flags = (FLAG_RECOMPUTE if recompute else 0) | (FLAG_LAYERNORM if layernorm else 0)
        self.shape = make_shape(tokens, hidden, ffn, t, dtype, algo, flags)
        if saved_bytes(self.shape) == 0 and tokens > 0:
            raise ValueError("invalid shape (tokens=%d hidden=%d ffn=%d t=%d)" % (tokens, hidden, ffn, t))
        self.dtype = dtype
        self.recompute = recompute
        dev = device or "cuda"
        self.H = torch.empty((tokens, ffn), dtype=dtype, device=dev) if (keep_H or recompute) else None
        self._Y = None if recompute else torch.empty((tokens, ffn), dtype=dtype, device=dev)
        self.workspace = new_workspace(self.shape, dev)
        self.saved = Saved(None, None, None, _ptr(self.H), _ptr(self._Y))
        self._keep = []
        if layernorm:
            self.Xn = torch.empty((tokens, hidden), dtype=dtype, device=dev)
            self.mean = torch.empty((tokens,), dtype=torch.float32, device=dev)
            self.rstd = torch.empty((tokens,), dtype=torch.float32, device=dev)
            self.ln = LayerNorm(None, None, None, _ptr(self.Xn), _ptr(self.mean), _ptr(self.rstd), float(eps))

    def _ws_view(self, region, cols=None):
        T = self.shape.tokens
        C = self.shape.ffn if cols is None else cols
        off = workspace_offset(self.shape, region)
        esz = 2 if self.dtype == torch.bfloat16 else 4
        return self.workspace[off:off + T * C * esz].view(self.dtype).view(T, C)

    @property
    def dXn(self) -> torch.Tensor:
        """The MLP's input gradient of the last sequence-parallel backward (the
        LayerNorm's output gradient; a view into the workspace)."""
        return self._ws_view(WS_DXN, self.shape.hidden)

    @property
    def Y(self) -> torch.Tensor:
        """GeLU(H): the caller-owned buffer, or under recomputation the workspace
        copy (written by forward, rebuilt by backward)."""
        return self._ws_view(WS_Y) if self.recompute else self._Y

    @property
    def dY(self) -> torch.Tensor:
        """The dY intermediate of the last backward (a view into the workspace)."""
        return self._ws_view(WS_DY)


def forward(ctx: Context, X, A, a, B, b, Z=None, stream=None, inference=False):
    """Z = GeLU(X A + a) B + b with the t-shard fold; fills ctx.H, ctx.Y.
    inference=True passes no saved record: nothing is kept for backward (Y goes
    to the workspace's dY region, H is not stored)."""
    s = ctx.shape
    T, h, F = s.tokens, s.hidden, s.ffn
    for x, n, shp in ((X, "X", (T, h)), (A, "A", (h, F)), (a, "a", (F,)), (B, "B", (F, h)), (b, "b", (h,))):
        _need(x, n, ctx.dtype, shp)
    if Z is None:
        Z = torch.empty((T, h), dtype=ctx.dtype, device=X.device)
    _need(Z, "Z", ctx.dtype, (T, h))
    ctx._keep = [X, A, B]
    st = lib.tpmlp_forward(ctypes.byref(s), _ptr(X), _ptr(A), _ptr(a), _ptr(B), _ptr(b), _ptr(Z),
                           None if inference else ctypes.byref(ctx.saved), _ptr(ctx.workspace), _stream(stream))
    _check(st, "tpmlp_forward")
    return Z


def backward(ctx: Context, dZ, dX=None, dA=None, da=None, dB=None, db=None, stream=None):
    """dX, dA, da, dB, db for L = sum(dZ * Z), using what forward saved in ctx."""
    s = ctx.shape
    T, h, F = s.tokens, s.hidden, s.ffn
    dev = dZ.device
    _need(dZ, "dZ", ctx.dtype, (T, h))
    out = {}
    for name, val, shp in (("dX", dX, (T, h)), ("dA", dA, (h, F)), ("da", da, (F,)),
                           ("dB", dB, (F, h)), ("db", db, (h,))):
        if val is None:
            val = torch.empty(shp, dtype=ctx.dtype, device=dev)
        _need(val, name, ctx.dtype, shp)
        out[name] = val
    st = lib.tpmlp_backward(ctypes.byref(s), _ptr(dZ), ctypes.byref(ctx.saved), _ptr(out["dX"]),
                            _ptr(out["dA"]), _ptr(out["da"]), _ptr(out["dB"]), _ptr(out["db"]),
                            _ptr(ctx.workspace), _stream(stream))
    _check(st, "tpmlp_backward")
    return out


def sp_forward(ctx: Context, X_in, gamma, beta, A, a, B, b, Z=None, stream=None):
    """Sequence-parallel block forward: Xn = LayerNorm(X_in), then the MLP on Xn."""
    s = ctx.shape
    T, h, F = s.tokens, s.hidden, s.ffn
    for x, n, shp in ((X_in, "X_in", (T, h)), (gamma, "gamma", (h,)), (beta, "beta", (h,)), (A, "A", (h, F)),
                      (a, "a", (F,)), (B, "B", (F, h)), (b, "b", (h,))):
        _need(x, n, ctx.dtype, shp)
    if Z is None:
        Z = torch.empty((T, h), dtype=ctx.dtype, device=X_in.device)
    _need(Z, "Z", ctx.dtype, (T, h))
    ctx.ln.X_in, ctx.ln.gamma, ctx.ln.beta = _ptr(X_in), _ptr(gamma), _ptr(beta)
    ctx._keep = [X_in, gamma, beta, A, B]
    st = lib.tpmlp_sp_forward(ctypes.byref(s), ctypes.byref(ctx.ln), _ptr(A), _ptr(a), _ptr(B), _ptr(b), _ptr(Z),
                              ctypes.byref(ctx.saved), _ptr(ctx.workspace), _stream(stream))
    _check(st, "tpmlp_sp_forward")
    return Z


def sp_backward(ctx: Context, dZ, stream=None, **outs):
    """Sequence-parallel block backward: dX_in, dgamma, dbeta and the MLP's
    weight and bias gradients."""
    s = ctx.shape
    T, h, F = s.tokens, s.hidden, s.ffn
    _need(dZ, "dZ", ctx.dtype, (T, h))
    out = {}
    for name, shp in (("dX_in", (T, h)), ("dgamma", (h,)), ("dbeta", (h,)), ("dA", (h, F)), ("da", (F,)),
                      ("dB", (F, h)), ("db", (h,))):
        val = outs.get(name)
        if val is None:
            val = torch.empty(shp, dtype=ctx.dtype, device=dZ.device)
        _need(val, name, ctx.dtype, shp)
        out[name] = val
    st = lib.tpmlp_sp_backward(ctypes.byref(s), ctypes.byref(ctx.ln), _ptr(dZ), ctypes.byref(ctx.saved),
                               *(_ptr(out[k]) for k in ("dX_in", "dgamma", "dbeta", "dA", "da", "dB", "db")),
                               _ptr(ctx.workspace), _stream(stream))
    _check(st, "tpmlp_sp_backward")
    return out


def ln_forward(ctx: Context, X_in, gamma, beta, stream=None):
    """LayerNorm alone (the block's first step): fills ctx.Xn, ctx.mean, ctx.rstd."""
    ctx.ln.X_in, ctx.ln.gamma, ctx.ln.beta = _ptr(X_in), _ptr(gamma), _ptr(beta)
    ctx._keep = [X_in, gamma, beta]
    _check(lib.tpmlp_ln_forward(ctypes.byref(ctx.shape), ctypes.byref(ctx.ln), _stream(stream)), "tpmlp_ln_forward")
    return ctx.Xn


def ln_backward(ctx: Context, dXn, stream=None):
    """LayerNorm backward alone for the gradient dXn of its output."""
    T, h = ctx.shape.tokens, ctx.shape.hidden
    dX_in = torch.empty((T, h), dtype=ctx.dtype, device=dXn.device)
    dg = torch.empty((h,), dtype=ctx.dtype, device=dXn.device)
    dbt = torch.empty((h,), dtype=ctx.dtype, device=dXn.device)
    st = lib.tpmlp_ln_backward(ctypes.byref(ctx.shape), ctypes.byref(ctx.ln), _ptr(dXn), _ptr(dX_in), _ptr(dg),
                               _ptr(dbt), _ptr(ctx.workspace), _stream(stream))
    _check(st, "tpmlp_ln_backward")
    return {"dX_in": dX_in, "dgamma": dg, "dbeta": dbt}


class AttnContext:
    """Buffers of one tensor-parallel self-attention layer between forward and
    backward: the saved QKV [T,3h], P [batch*heads, seq, seq], O [T,h] and the
    workspace (bf16 only).

    p_upper_zero=True (the default) allocates P zeroed and sets
    ATTN_P_UPPER_ZERO: the tiles of P wholly above the diagonal keep those
    zeros and the forward does not rewrite them.  False: P is allocated
    uninitialised and every row is written in full."""

    def __init__(self, batch, seq, hidden, heads, t, device=None, p_upper_zero=True):
        flags = ATTN_P_UPPER_ZERO if p_upper_zero else 0
        self.shape = AttnShape(int(batch), int(seq), int(hidden), int(heads), int(t), BF16, flags)
        n = int(lib.tpmlp_attn_workspace_bytes(ctypes.byref(self.shape)))
        if n == 0:
            raise ValueError("invalid attention shape (batch=%d seq=%d hidden=%d heads=%d t=%d)"
                             % (batch, seq, hidden, heads, t))
        dev = device or "cuda"
        T, h = batch * seq, hidden
        self.dtype = torch.bfloat16
        self.QKV = torch.empty((T, 3 * h), dtype=self.dtype, device=dev)
        alloc = torch.zeros if p_upper_zero else torch.empty
        self.P = alloc((batch * heads, seq, seq), dtype=self.dtype, device=dev)
        self.O = torch.empty((T, h), dtype=self.dtype, device=dev)
        self.workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
        self.saved = AttnSaved(None, None, None, _ptr(self.QKV), _ptr(self.P), _ptr(self.O))
        self._keep = []

    @property
    def tokens(self) -> int:
        return self.shape.batch * self.shape.seq


def attn_saved_bytes(batch, seq, hidden, heads, t) -> int:
    s = AttnShape(int(batch), int(seq), int(hidden), int(heads), int(t), BF16, 0)
    return int(lib.tpmlp_attn_saved_bytes(ctypes.byref(s)))


def attn_forward(ctx: AttnContext, X, Wqkv, bqkv, Wo, bo, Z=None, stream=None):
    """Z = bo + sum_i O_i Wo_i with per-head causal attention over X Wqkv + bqkv."""
    s = ctx.shape
    T, h = ctx.tokens, s.hidden
    for x, n, shp in ((X, "X", (T, h)), (Wqkv, "Wqkv", (h, 3 * h)), (bqkv, "bqkv", (3 * h,)),
                      (Wo, "Wo", (h, h)), (bo, "bo", (h,))):
        _need(x, n, ctx.dtype, shp)
    if Z is None:
        Z = torch.empty((T, h), dtype=ctx.dtype, device=X.device)
    _need(Z, "Z", ctx.dtype, (T, h))
    ctx._keep = [X, Wqkv, Wo]
    st = lib.tpmlp_attn_forward(ctypes.byref(s), _ptr(X), _ptr(Wqkv), _ptr(bqkv), _ptr(Wo), _ptr(bo), _ptr(Z),
                                ctypes.byref(ctx.saved), _ptr(ctx.workspace), _stream(stream))
    _check(st, "tpmlp_attn_forward")
    return Z


def attn_backward(ctx: AttnContext, dZ, stream=None, **outs):
    """dX, dWqkv, dbqkv, dWo, dbo for L = sum(dZ * Z), from what attn_forward saved."""
    s = ctx.shape
    T, h = ctx.tokens, s.hidden
    _need(dZ, "dZ", ctx.dtype, (T, h))
    out = {}
    for name, shp in (("dX", (T, h)), ("dWqkv", (h, 3 * h)), ("dbqkv", (3 * h,)), ("dWo", (h, h)),
                      ("dbo", (h,))):
        val = outs.get(name)
        if val is None:
            val = torch.empty(shp, dtype=ctx.dtype, device=dZ.device)
        _need(val, name, ctx.dtype, shp)
        out[name] = val
    st = lib.tpmlp_attn_backward(ctypes.byref(s), _ptr(dZ), ctypes.byref(ctx.saved),
                                 *(_ptr(out[k]) for k in ("dX", "dWqkv", "dbqkv", "dWo", "dbo")),
                                 _ptr(ctx.workspace), _stream(stream))
    _check(st, "tpmlp_attn_backward")
    return out


def _status_workspace(nbytes, device):
    """A workspace whose status word is zero; the rest is written before it is read."""
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    ws[:1024].zero_()
    return ws


def _same_device(ctx, *tensors):
    device = ctx.workspace.device
    for x in tensors:
        if x is not None and x.device != device:
            raise ValueError("tensor on %s, the context's workspace on %s" % (x.device, device))


# The current stream's handle without a Stream object around it, where this PyTorch has it
# (a tenth of the time, and calls on small inputs are bound by the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# A context's workspace exists, so CUDA is up: the current device without a check for that.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(ctx, fn, name, args, stream):
    """fn(*args, stream) with the context's device as the current one."""
    index = ctx.workspace.device.index
    if index != _current_device():
        with torch.cuda.device(index):
            _check(fn(*args, _stream(stream)), name)
    elif stream is None and _raw_stream is not None:
        _check(fn(*args, _raw_stream(index)), name)
    else:
        _check(fn(*args, _stream(stream)), name)


class XentContext:
    """Buffers of the vocabulary cross entropy between forward and backward: lse [T]
    (fp32) and the workspace.  W is [vocab, hidden], targets are int64; a target equal
    to ignore_index takes no part.  `piece` sets the vocabulary rows per piece of the
    backward pass (a multiple of 8; 0: the library's choice).  backward=False is for scoring
    alone: the workspace then holds the forward pass only, and xent_backward is refused.

    One context serves one call at a time: its workspace is scratch of every call,
    also of captured graphs replayed at the same time."""

    def __init__(self, tokens, hidden, vocab, dtype, ignore_index=-100, piece=0, algo=ALGO_DEFAULT, device=None,
                 backward=True):
        if dtype not in _DTYPES:
            raise ValueError("dtype %s: float32 or bfloat16" % (dtype,))
        self.shape = XentShape(int(tokens), int(hidden), int(vocab), int(ignore_index), int(piece), _DTYPES[dtype],
                               int(algo))
        size = lib.tpmlp_xent_workspace_bytes if backward else lib.tpmlp_xent_forward_workspace_bytes
        n = int(size(ctypes.byref(self.shape)))
        if n == 0:
            raise ValueError("invalid cross entropy shape (tokens=%d hidden=%d vocab=%d piece=%d)"
                             % (tokens, hidden, vocab, piece))
        self.dtype = dtype
        self.backward = bool(backward)
        self.workspace = _status_workspace(n, device)
        self.lse = torch.empty((int(tokens),), dtype=torch.float32, device=self.workspace.device)
        self._saved = None


def xent_forward(ctx: XentContext, X, W, target, loss=None, stream=None, lse=None):
    """loss[T] = log sum_v exp(X W^T)_v - (X W^T)_target, 0 for an ignored target.  The log of
    the sum goes to `lse` [T] (fp32), or without it to ctx.lse, which the next call overwrites.
    X, W, target and the lse are kept, not copied, for xent_backward: they have to hold the same
    values then."""
    s = ctx.shape
    T, h, V = s.tokens, s.hidden, s.vocab
    _need(X, "X", ctx.dtype, (T, h))
    _need(W, "W", ctx.dtype, (V, h))
    _need(target, "target", torch.int64, (T,))
    if loss is None:
        loss = torch.empty((T,), dtype=torch.float32, device=X.device)
    _need(loss, "loss", torch.float32, (T,))
    if lse is None:
        lse = ctx.lse
    else:
        _need(lse, "lse", torch.float32, (T,))
    _same_device(ctx, X, W, target, loss, lse)
    _call(ctx, lib.tpmlp_xent_forward, "tpmlp_xent_forward",
          (ctypes.byref(s), X.data_ptr(), W.data_ptr(), target.data_ptr(), loss.data_ptr(), lse.data_ptr(),
           ctx.workspace.data_ptr()), stream)
    ctx._saved = (X, W, target, lse)
    return loss


def xent_backward(ctx: XentContext, dloss, dX=None, dW=None, need_dX=True, need_dW=True, stream=None):
    """dX[T,h] and dW[V,h] for the gradients dloss[T] (fp32) of the losses that the
    last xent_forward of this context returned; need_dX=False or need_dW=False leaves
    one out (its entry is None)."""
    if not ctx.backward:
        raise ValueError("xent_backward of a context made with backward=False")
    if ctx._saved is None:
        raise ValueError("xent_backward needs an xent_forward of the same context before it")
    X, W, target, lse = ctx._saved
    s = ctx.shape
    T, h, V = s.tokens, s.hidden, s.vocab
    _need(dloss, "dloss", torch.float32, (T,))
    if need_dX and dX is None:
        dX = torch.empty((T, h), dtype=ctx.dtype, device=X.device)
    if need_dW and dW is None:
        dW = torch.empty((V, h), dtype=ctx.dtype, device=X.device)
    dX, dW = dX if need_dX else None, dW if need_dW else None
    for x, n, shp in ((dX, "dX", (T, h)), (dW, "dW", (V, h))):
        if x is not None:
            _need(x, n, ctx.dtype, shp)
    _same_device(ctx, dloss, dX, dW)
    _call(ctx, lib.tpmlp_xent_backward, "tpmlp_xent_backward",
          (ctypes.byref(s), X.data_ptr(), W.data_ptr(), target.data_ptr(), lse.data_ptr(), dloss.data_ptr(),
           _ptr(dX), _ptr(dW), ctx.workspace.data_ptr()), stream)
    return {"dX": dX, "dW": dW}


class OrthoContext:
    """Workspace of the Newton-Schulz orthogonalisation of `batch` matrices [rows, cols]
    of the given dtype (float32 or bfloat16; the output is bfloat16): `steps` steps of
    X <- a X + (b A + c A^2) X with A = X X^T, from X = G / (|G| + eps).

    One context serves one call at a time (see XentContext)."""

    def __init__(self, rows, cols, batch=1, dtype=torch.bfloat16, steps=5, coefficients=(3.4445, -4.7750, 2.0315),
                 eps=1e-7, device=None):
        if dtype not in _DTYPES:
            raise ValueError("dtype %s: float32 or bfloat16" % (dtype,))
        a, b, c = coefficients
        self.shape = OrthoShape(int(batch), int(rows), int(cols), int(steps), _DTYPES[dtype], a, b, c, eps)
        n = int(lib.tpmlp_ortho_workspace_bytes(ctypes.byref(self.shape)))
        if n == 0:
            raise ValueError("invalid orthogonalisation shape (batch=%d rows=%d cols=%d steps=%d eps=%g)"
                             % (batch, rows, cols, steps, eps))
        self.dtype = dtype
        self.workspace = _status_workspace(n, device)


def orthogonalize(ctx: OrthoContext, G, O=None, stream=None):
    """O (bfloat16) from G, both [batch, rows, cols], or [rows, cols] where batch is 1."""
    s = ctx.shape
    shape = (s.batch, s.rows, s.cols)
    if s.batch == 1 and G.dim() == 2:
        shape = shape[1:]
    _need(G, "G", ctx.dtype, shape)
    if O is None:
        O = torch.empty(shape, dtype=torch.bfloat16, device=G.device)
    _need(O, "O", torch.bfloat16, shape)
    _same_device(ctx, G, O)
    _call(ctx, lib.tpmlp_orthogonalize, "tpmlp_orthogonalize",
          (ctypes.byref(s), G.data_ptr(), O.data_ptr(), ctx.workspace.data_ptr()), stream)
    return O


class RopeTable:
    """The rotation of positions: the first `rot` components of a head in pairs (i, i + rot/2) ("half") or
    (2i, 2i + 1) ("interleaved"), pair i by position * base^(-2i/rot).

    scaling stretches it to contexts longer than the trained one: ("linear", factor), or
    ("parts", factor, context, low, high): pairs that turn `high` times or more within the trained context
    keep their angles, those that turn `low` times or less are divided by factor, the others in between.
    amplitude multiplies the rotated components."""

    def __init__(self, rot, base=10000.0, layout="half", scaling=None, amplitude=1.0, device=None):
        kinds = {"linear": ROPE_SCALE_LINEAR, "parts": ROPE_SCALE_PARTS}
        layouts = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED}
        if layout not in layouts:
            raise ValueError("layout %r: 'half' or 'interleaved'" % (layout,))
        if scaling is not None and (scaling[0] not in kinds or len(scaling) != (2 if scaling[0] == "linear" else 5)):
            raise ValueError("scaling %r: ('linear', factor) or ('parts', factor, context, low, high)" % (scaling,))
        kind, factor, context, low, high = (tuple(scaling or (None,)) + (1.0, 1, 0.0, 1.0)[len(scaling or (None,)) - 1:])
        rope = Rope(float(base), float(factor), float(low), float(high), int(context), int(rot),
                    kinds.get(kind, ROPE_SCALE_NONE))
        turns = (ctypes.c_uint64 * max(rope.rot // 2, 1))()
        _check(lib.tpmlp_rope_turns(ctypes.byref(rope), turns), "tpmlp_rope_turns")
        self.rot, self.layout, self.amplitude = rope.rot, layouts[layout], float(amplitude)
        self.turns = torch.tensor([x - (1 << 64) if x >> 63 else x for x in turns], dtype=torch.int64,
                                  device=device or "cuda")


class QkContext:
    """Norms of queries and keys per head and their rotation, for `tokens` tokens of the attention block's
    projection: `heads` query heads and `kv_heads` key and value heads of `dim` components, the columns of QKV
    shard-major in t shards [Q_1 | K_1 | V_1 | Q_2 | ...].  rope: a RopeTable, or None for the norm alone;
    norm=False: the rotation alone.  eps is the norm's.

    QKV is [tokens, (heads + 2 kv_heads) dim] (its rows may be apart), or a tuple (Q, K) or (Q, K, V) of
    [tokens, heads, dim] tensors, shards' heads one after another.

    One context serves one call at a time (see XentContext)."""

    def __init__(self, tokens, heads, kv_heads, dim, dtype, rope=None, norm=True, eps=1e-6, t=1, device=None):
        if dtype not in _DTYPES:
            raise ValueError("dtype %s: float32 or bfloat16" % (dtype,))
        self.shape = QkShape(int(tokens), int(heads), int(kv_heads), int(dim), int(t), _DTYPES[dtype],
                             rope.layout if rope else ROPE_HALF, rope.rot if rope else 0, 1 if norm else 0, float(eps),
                             rope.amplitude if rope else 1.0)
        n = int(lib.tpmlp_qk_workspace_bytes(ctypes.byref(self.shape)))
        if n == 0:
            raise ValueError("invalid shape (tokens=%d heads=%d kv_heads=%d dim=%d rot=%d t=%d eps=%g)"
                             % (tokens, heads, kv_heads, dim, self.shape.rot, t, eps))
        self.dtype = dtype
        self.rope = rope
        self.workspace = _status_workspace(n, device)
        if rope is not None and rope.turns.device != self.workspace.device:
            raise ValueError("rope table on %s, the context's workspace on %s" % (rope.turns.device, self.workspace.device))
        self._turns = rope.turns.data_ptr() if rope else None
        self._saved = None
        # the C ABI's records, filled in at every call: Q, K, V, two outputs, two gradients
        self._records = [Heads() for _ in range(7)]
        self._refs = [ctypes.byref(r) for r in self._records]
        self._shape_ref = ctypes.byref(self.shape)
        s = self.shape
        self._tokens, self._heads, self._kv_heads, self._dim = s.tokens, s.heads, s.kv_heads, s.dim
        self._q_width, self._k_width = s.heads // s.t * s.dim, s.kv_heads // s.t * s.dim  # of a shard
        self._qkv_shape = (s.tokens, s.t * (self._q_width + 2 * self._k_width))
        self._rot, self._norm, self._device = s.rot, s.norm, self.workspace.device


def _on_device(ctx, x, name):
    if x.dtype is not ctx.dtype or not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor of %s" % (name, ctx.dtype))
    if x.device != ctx._device:
        raise ValueError("tensor on %s, the context's workspace on %s" % (x.device, ctx._device))


def _dense_heads(ctx, record, x, heads, name):
    """A [tokens, heads, dim] tensor whose heads follow one another; its rows may be apart."""
    _on_device(ctx, x, name)
    if x.shape != (ctx._tokens, heads, ctx._dim):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(x.shape), (ctx._tokens, heads, ctx._dim)))
    row, head, one = x.stride()
    if (one != 1 or (heads > 1 and head != ctx._dim)) and x.numel():
        raise ValueError("%s: a token's heads must be contiguous" % name)
    record.p, record.row = x.data_ptr(), row
    record.shard = ctx._q_width if heads == ctx._heads else ctx._k_width


def _qkv_heads(ctx, records, x, name):
    """Q, K and V (three records) or Q and K (two) inside a projection's array."""
    _on_device(ctx, x, name)
    if x.shape != ctx._qkv_shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(x.shape), ctx._qkv_shape))
    row, one = x.stride()
    if one != 1 and x.numel():
        raise ValueError("%s: a token's columns must be contiguous" % name)
    p, e, n, m = x.data_ptr(), 2 if ctx.dtype is torch.bfloat16 else 4, ctx._q_width, ctx._k_width
    shard, off = n + 2 * m, 0
    for r in records:
        r.p, r.row, r.shard = p + off * e, row, shard
        off = off + m if off else n


def _qkv_input(ctx, QKV, values):
    if isinstance(QKV, torch.Tensor):
        _qkv_heads(ctx, ctx._records[:3 if values else 2], QKV, "QKV")
        return
    if len(QKV) < (3 if values else 2):
        raise ValueError("Q, K%s expected" % (" and V" if values else ""))
    for r, x, n, name in zip(ctx._records, QKV, (ctx._heads, ctx._kv_heads, ctx._kv_heads), ("Q", "K", "V")):
        _dense_heads(ctx, r, x, n, name)


def _qk_inputs(ctx, position, gain_q, gain_k):
    p = q = k = None
    if ctx._rot:
        _need(position, "position", torch.int64, (ctx._tokens,))
        _same_device(ctx, position)
        p = position.data_ptr()
    if ctx._norm:
        _need(gain_q, "gain_q", ctx.dtype, (ctx._dim,))
        _need(gain_k, "gain_k", ctx.dtype, (ctx._dim,))
        _same_device(ctx, gain_q, gain_k)
        q, k = gain_q.data_ptr(), gain_k.data_ptr()
    return q, k, p, ctx._turns


def _new_heads(ctx, record, heads):
    x = torch.empty((ctx._tokens, heads, ctx._dim), dtype=ctx.dtype, device=ctx._device)
    record.p, record.row = x.data_ptr(), heads * ctx._dim
    record.shard = ctx._q_width if heads == ctx._heads else ctx._k_width
    return x


def _qk_out(ctx, out, names):
    """The output's records; without one, dense tensors."""
    records = ctx._records
    if out is None:
        return _new_heads(ctx, records[3], ctx._heads), _new_heads(ctx, records[4], ctx._kv_heads)
    if isinstance(out, torch.Tensor):
        _qkv_heads(ctx, records[3:5], out, "out")
        return out
    for r, x, n, name in zip(records[3:5], out, (ctx._heads, ctx._kv_heads), names):
        _dense_heads(ctx, r, x, n, name)
    return tuple(out)


def qk_forward(ctx: QkContext, QKV, position, gain_q=None, gain_k=None, out=None, stream=None):
    """(Qr, Kr) from QKV's queries and keys: normed (gains [dim]) and rotated by position [tokens] (int64).
    out: a tuple of [tokens, heads, dim] tensors, or an array laid out as QKV whose Q and K columns are
    written (QKV itself: in place) and which is then returned.  QKV, position and gains are kept, not
    copied, for qk_backward: they have to hold the same values then."""
    ctx._saved = None  # (a call that is refused leaves no earlier pass to go back from)
    _qkv_input(ctx, QKV, False)
    given = _qk_inputs(ctx, position, gain_q, gain_k)
    result = _qk_out(ctx, out, ("Qr", "Kr"))
    r, records = ctx._refs, ctx._records
    _call(ctx, lib.tpmlp_qk_forward, "tpmlp_qk_forward", (ctx._shape_ref, r[0], r[1], *given, r[3], r[4]), stream)
    q, k = records[0], records[1]
    kept = not (ctx._norm and ctx._tokens) or (q.p != records[3].p and k.p != records[4].p)
    # the tensors are kept so that what the records point to stays
    ctx._saved = ((QKV, position, gain_q, gain_k), (q.p, q.row, q.shard), (k.p, k.row, k.shard), given) if kept else ()
    return result


def _written_over(ctx, *outputs):
    """An output in the place of the saved Q or K, which a backward pass with the norm reads: there is no other one."""
    if ctx._saved and ctx._norm and ctx._tokens:
        q, k = ctx._saved[1][0], ctx._saved[2][0]
        if any(r.p == q or r.p == k for r in outputs):
            ctx._saved = ()


def qk_backward(ctx: QkContext, dQr, dKr, out=None, dgain_q=None, dgain_k=None, stream=None):
    """{"dQ", "dK", "dgain_q", "dgain_k"} from the gradients of what the last qk_forward of this context returned
    ([tokens, heads, dim] each).  out: as for qk_forward (an array laid out as QKV is returned as "dQKV"); it may be
    what holds dQr and dKr, or the QKV of the forward pass: with the norm there is no second backward pass then.  The
    gains' entries are None without the norm."""
    if ctx._saved is None:
        raise ValueError("qk_backward needs a qk_forward of the same context before it")
    if not ctx._saved:
        raise ValueError("qk_backward after a pass with the norm that wrote in place of its inputs: they are gone")
    _, q, k, given = ctx._saved
    records, r = ctx._records, ctx._refs
    records[0].p, records[0].row, records[0].shard = q
    records[1].p, records[1].row, records[1].shard = k
    _dense_heads(ctx, records[5], dQr, ctx._heads, "dQr")
    _dense_heads(ctx, records[6], dKr, ctx._kv_heads, "dKr")
    result = _qk_out(ctx, out, ("dQ", "dK"))
    to_q = to_k = None
    if ctx._norm:
        if dgain_q is None:
            dgain_q = torch.empty((ctx._dim,), dtype=ctx.dtype, device=ctx._device)
        else:
            _need(dgain_q, "dgain_q", ctx.dtype, (ctx._dim,))
        if dgain_k is None:
            dgain_k = torch.empty((ctx._dim,), dtype=ctx.dtype, device=ctx._device)
        else:
            _need(dgain_k, "dgain_k", ctx.dtype, (ctx._dim,))
        _same_device(ctx, dgain_q, dgain_k)
        to_q, to_k = dgain_q.data_ptr(), dgain_k.data_ptr()
    else:
        dgain_q = dgain_k = None
    _call(ctx, lib.tpmlp_qk_backward, "tpmlp_qk_backward",
          (ctx._shape_ref, r[0], r[1], *given, r[5], r[6], r[3], r[4], to_q, to_k, ctx.workspace.data_ptr()), stream)
    _written_over(ctx, records[3], records[4])
    grads = {"dgain_q": dgain_q, "dgain_k": dgain_k}
    if isinstance(result, torch.Tensor):
        grads["dQKV"] = result
    else:
        grads["dQ"], grads["dK"] = result
    return grads


class KvCache:
    """Keys and values of many sequences in pages of page_size tokens: K and V [pages, kv_heads, page_size, dim].
    KvCache.of(K, V) takes existing tensors of that shape, of any strides that keep a row's components together
    (a [pages, page_size, kv_heads, dim] cache is K.transpose(1, 2))."""

    def __init__(self, pages, page_size, kv_heads, dim, dtype, device=None):
        shape = (int(pages), int(kv_heads), int(page_size), int(dim))
        self._set(*(torch.zeros(shape, dtype=dtype, device=device or "cuda") for _ in "kv"))

    @classmethod
    def of(cls, K, V):
        self = cls.__new__(cls)
        self._set(K, V)
        return self

    def _set(self, K, V):
        if K.dtype not in _DTYPES or V.dtype is not K.dtype:
            raise ValueError("K %s and V %s: float32 or bfloat16, the same" % (K.dtype, V.dtype))
        if not (K.is_cuda and V.device == K.device) or K.dim() != 4 or V.shape != K.shape:
            raise ValueError("K and V must be CUDA tensors [pages, kv_heads, page_size, dim] of one device")
        if V.stride() != K.stride() or K.stride(3) != 1:
            raise ValueError("K and V must have the same strides, and a row's components follow one another")
        self.K, self.V, self.dtype = K, V, K.dtype
        pages, kv_heads, page_size, dim = K.shape
        self.shape = KvCacheShape(K.data_ptr(), V.data_ptr(), pages, page_size, K.stride(0), K.stride(1), K.stride(2),
                                  kv_heads, dim, _DTYPES[K.dtype])
        self.kv_heads, self.dim = kv_heads, dim
        self._ref = ctypes.byref(self.shape)


def kv_append(ctx: QkContext, cache: KvCache, QKV, position, slot, gain_q=None, gain_k=None, out=None, stream=None):
    """Puts the tokens' keys (normed, rotated) and values at slot [tokens] (int64: page * page_size + row, each
    once; negative: not kept) of the cache, and returns their queries, normed and rotated, [tokens, heads, dim] (`out`, where given)."""
    _qkv_input(ctx, QKV, True)
    given = _qk_inputs(ctx, position, gain_q, gain_k)
    _need(slot, "slot", torch.int64, (ctx._tokens,))
    _same_device(ctx, slot, cache.K)
    if out is None:
        out = _new_heads(ctx, ctx._records[3], ctx._heads)
    else:
        _dense_heads(ctx, ctx._records[3], out, ctx._heads, "out")
    r = ctx._refs
    _call(ctx, lib.tpmlp_kv_append, "tpmlp_kv_append",
          (ctx._shape_ref, cache._ref, r[0], r[1], r[2], *given, slot.data_ptr(), r[3], ctx.workspace.data_ptr()), stream)
    _written_over(ctx, ctx._records[3])
    return out


class CacheAttnContext:
    """Workspace of attention over a paged cache: `tokens` new tokens of `batch` sequences, `heads` query heads over the
    cache's kv_heads.  scale: of the scores, 1/sqrt(dim) where it is None.  The number of pages per sequence and
    of a tree's words may differ from call to call.

    One context serves one call at a time (see XentContext)."""

    def __init__(self, tokens, batch, heads, kv_heads, dim, dtype, scale=None, algo=ALGO_DEFAULT, device=None):
        if dtype not in _DTYPES:
            raise ValueError("dtype %s: float32 or bfloat16" % (dtype,))
        self.shape = CacheAttnShape(int(tokens), int(batch), 0, int(heads), 0, int(algo),
                                    float(dim) ** -0.5 if scale is None else float(scale))
        sizes = KvCacheShape(None, None, 1, 1, int(dim) * int(kv_heads), int(dim), int(dim) * int(kv_heads), int(kv_heads),
                             int(dim), _DTYPES[dtype])
        n = int(lib.tpmlp_cache_attn_workspace_bytes(ctypes.byref(self.shape), ctypes.byref(sizes)))
        if n == 0:
            raise ValueError("invalid shape (tokens=%d batch=%d heads=%d kv_heads=%d dim=%d scale=%g)"
                             % (tokens, batch, heads, kv_heads, dim, self.shape.scale))
        self.dtype, self.kv_heads, self.dim = dtype, int(kv_heads), int(dim)
        self._tokens, self._batch, self._heads = int(tokens), int(batch), int(heads)
        self.workspace = _status_workspace(n, device)
        self._ref = ctypes.byref(self.shape)


def cache_attention(ctx: CacheAttnContext, cache: KvCache, Q, q_start, kv_len, page_table, tree=None, O=None, stream=None):
    """O [tokens, heads, dim]: attention of Q over the cache, which holds the new tokens' keys already.  Sequence b has
    tokens q_start[b] .. q_start[b+1] - 1 and kv_len[b] keys in the pages page_table[b] (all int32); its new tokens are the
    last of those keys, and each sees the keys before them, and of the new ones those up to itself, or with tree
    [tokens, words] (int64) those whose bit is set."""
    if cache.dtype is not ctx.dtype or cache.kv_heads != ctx.kv_heads or cache.dim != ctx.dim:
        raise ValueError("the cache has %s, %d heads of %d; the context %s, %d of %d"
                         % (cache.dtype, cache.kv_heads, cache.dim, ctx.dtype, ctx.kv_heads, ctx.dim))
    s, T, batch, shape = ctx.shape, ctx._tokens, ctx._batch, (ctx._tokens, ctx._heads, ctx.dim)
    _need(Q, "Q", ctx.dtype, shape)
    _need(q_start, "q_start", torch.int32, (batch + 1,))
    _need(kv_len, "kv_len", torch.int32, (batch,))
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, pages]")
    _need(page_table, "page_table", torch.int32, (batch, page_table.shape[1]))
    if tree is not None:
        if tree.dim() != 2 or tree.shape[1] == 0:
            raise ValueError("tree must be [tokens, words] with a word at least")
        _need(tree, "tree", torch.int64, (T, tree.shape[1]))
    if O is None:
        O = torch.empty_like(Q)
    else:
        _need(O, "O", ctx.dtype, shape)
    _same_device(ctx, Q, q_start, kv_len, page_table, tree, O, cache.K)
    s.max_pages, s.tree_words = page_table.shape[1], 0 if tree is None else tree.shape[1]
    _call(ctx, lib.tpmlp_cache_attn, "tpmlp_cache_attn",
          (ctx._ref, cache._ref, Q.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(),
           None if tree is None else tree.data_ptr(), O.data_ptr(), ctx.workspace.data_ptr()), stream)
    return O


def check_device_status(ctx_or_ws, stream=None) -> int:
    known = (Context, AttnContext, XentContext, OrthoContext, QkContext, CacheAttnContext)
    ws = ctx_or_ws.workspace if isinstance(ctx_or_ws, known) else ctx_or_ws
    return int(lib.tpmlp_check_device_status(_ptr(ws), _stream(stream)))


def set_wait_limit_ns(ns: int):
    lib.tpmlp_set_wait_limit_ns(int(ns))


def debug_timeout_probe(workspace, wait_ns: int, stream=None) -> int:
    return int(lib.tpmlp_debug_timeout_probe(_ptr(workspace), int(wait_ns), _stream(stream)))


def launch_count() -> int:
    return int(lib.tpmlp_launch_count())


def profile_enable(on: bool = True):
    lib.tpmlp_profile_enable(1 if on else 0)


def profile_reset():
    lib.tpmlp_profile_reset()


def profile_collect() -> dict:
    """{kernel name: (launches, total ms)} of the launches timed since the reset."""
    _check(lib.tpmlp_profile_collect(), "tpmlp_profile_collect")
    out = {}
    buf = ctypes.create_string_buffer(128)
    for i in range(lib.tpmlp_profile_count()):
        n = ctypes.c_int64()
        ms = ctypes.c_double()
        if lib.tpmlp_profile_entry(i, buf, 128, ctypes.byref(n), ctypes.byref(ms)) == 0:
            out[buf.value.decode()] = (int(n.value), float(ms.value))
    return out
