"""Host side of the norms, the rotation and the paged cache, without a GPU: sizes, angles, argument checks that fail
before any CUDA call (no pointer is ever dereferenced), and the arithmetic that shares the tiles out, restated."""
import ctypes
import itertools
import math
import random

import pytest

FAKE = 1 << 44  # never dereferenced


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import build
    build.build()
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


ref = ctypes.byref


def qshape(tp, T=16, heads=8, kv=2, dim=64, t=1, dtype=None, layout=0, rot=64, norm=1, eps=1e-6, amplitude=1.0):
    return tp.QkShape(T, heads, kv, dim, t, tp.BF16 if dtype is None else dtype, layout, rot, norm, eps, amplitude)


def cshape(tp, K=FAKE, V=FAKE + (1 << 34), pages=8, page=16, kv=2, dim=64, dtype=None, strides=None):
    ps, hs, ts = strides or (kv * page * dim, page * dim, dim)
    return tp.KvCacheShape(K, V, pages, page, ps, hs, ts, kv, dim, tp.BF16 if dtype is None else dtype)


def ashape(tp, T=16, batch=3, max_pages=4, heads=8, words=0, algo=0, scale=0.125):
    return tp.CacheAttnShape(T, batch, max_pages, heads, words, algo, scale)


# ---- angles ---------------------------------------------------------------------------------------

def turns(tp, **kw):
    a = dict(base=10000.0, factor=1.0, low=0.0, high=1.0, context=1, rot=64, scaling=0)
    a.update(kw)
    r = tp.Rope(a["base"], a["factor"], a["low"], a["high"], a["context"], a["rot"], a["scaling"])
    out = (ctypes.c_uint64 * max(1, a["rot"] // 2))()
    return tp.lib.tpmlp_rope_turns(ref(r), out), list(out)[:max(0, a["rot"] // 2)]


@pytest.mark.parametrize("rot", [2, 64, 96, 256])
@pytest.mark.parametrize("base", [1.5, 10000.0, 5e5])
def test_turns(tp, rot, base):
    """theta / (2 pi) in units of 2^-64, cut off to whole ones: the power and the quotient are off by a few 2^-53 each."""
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    stretched = []
    for f in plain:
        n = 4096 * f / (2 * math.pi)
        k = min(1.0, max(0.0, (n - 1.0) / (32.0 - 1.0)))
        stretched.append(f * (k + (1 - k) / 8))
    for kw, want in ((dict(), plain), (dict(scaling=tp.ROPE_SCALE_LINEAR, factor=4.0), [f / 4 for f in plain]),
                     (dict(scaling=tp.ROPE_SCALE_PARTS, factor=8.0, context=4096, low=1.0, high=32.0), stretched)):
        status, got = turns(tp, rot=rot, base=base, **kw)
        assert status == tp.OK
        for g, f in zip(got, want):
            assert abs(g / 2 ** 64 - f / (2 * math.pi)) <= 2.0 ** -48 * f + 2.0 ** -64


def test_turns_are_refused(tp):
    assert tp.lib.tpmlp_rope_turns(None, None) == tp.ERR_INVALID_ARG
    nan, inf = float("nan"), float("inf")
    linear, parts = tp.ROPE_SCALE_LINEAR, tp.ROPE_SCALE_PARTS
    good = dict(scaling=parts, factor=2.0, low=1.0, high=4.0, context=2048)
    assert turns(tp, **good)[0] == tp.OK and turns(tp, rot=0)[0] == tp.OK
    for bad in (dict(rot=3), dict(rot=-2), dict(rot=258), dict(base=0.5), dict(base=nan), dict(base=inf), dict(scaling=9),
                dict(scaling=linear, factor=0.0), dict(scaling=linear, factor=-1.0), dict(scaling=linear, factor=nan),
                dict(scaling=linear, factor=inf), dict(scaling=linear, factor=0.1),  # more than a turn per position
                dict(good, factor=0.0), dict(good, low=4.0), dict(good, high=nan), dict(good, high=inf), dict(good, context=0)):
        if bad.get("rot", 64) in (3, -2, 258):
            r = tp.Rope(10000.0, 1.0, 0.0, 1.0, 1, bad["rot"], 0)
            assert tp.lib.tpmlp_rope_turns(ref(r), (ctypes.c_uint64 * 256)()) == tp.ERR_INVALID_ARG
        else:
            assert turns(tp, **bad)[0] == tp.ERR_INVALID_ARG, bad


# ---- norms and rotation -----------------------------------------------------------------------------

BAD_QK = (dict(T=-1), dict(T=(1 << 30) + 1), dict(heads=0), dict(kv=0), dict(heads=65537), dict(t=0), dict(t=17), dict(t=3),
          dict(t=4), dict(dim=0), dict(dim=63), dict(dim=258), dict(rot=63), dict(rot=66), dict(rot=-2), dict(dtype=5), dict(layout=2),
          dict(norm=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(amplitude=float("nan")))


def test_qk_workspace(tp):
    size = lambda **k: tp.lib.tpmlp_qk_workspace_bytes(ref(qshape(tp, **k)))
    assert size(T=0) >= 1024 and size() >= 1024 and size(T=1 << 30) < 64 << 20
    assert tp.lib.tpmlp_qk_workspace_bytes(None) == 0
    for bad in BAD_QK:
        assert size(**bad) == 0, bad


class Qk:
    """One call's arguments; arrays far apart, unless a test moves them."""

    def __init__(self, tp, **kw):
        self.tp, self.s = tp, qshape(tp, **kw)
        s = self.s
        self.h = {}
        for i, (name, n) in enumerate((("q", s.heads), ("k", s.kv_heads), ("v", s.kv_heads), ("oq", s.heads), ("ok", s.kv_heads),
                                       ("dq", s.heads), ("dk", s.kv_heads))):
            self.h[name] = tp.Heads(FAKE + (i << 34), n * s.dim, n // s.t * s.dim if s.t else 0)
        self.p = {x: FAKE + (16 + i << 34) for i, x in enumerate(("gq", "gk", "pos", "turns", "dgq", "dgk", "ws", "slot"))}
        self.cache = cshape(tp, FAKE + (30 << 34), FAKE + (31 << 34))

    def r(self, name):
        h = self.h[name]
        return None if h is None else ref(h)

    def forward(self):
        p = self.p
        return self.tp.lib.tpmlp_qk_forward(ref(self.s), self.r("q"), self.r("k"), p["gq"], p["gk"], p["pos"], p["turns"],
                                            self.r("oq"), self.r("ok"), None)

    def backward(self):
        p = self.p
        return self.tp.lib.tpmlp_qk_backward(ref(self.s), self.r("q"), self.r("k"), p["gq"], p["gk"], p["pos"], p["turns"],
                                             self.r("dq"), self.r("dk"), self.r("oq"), self.r("ok"), p["dgq"], p["dgk"], p["ws"], None)

    def append(self):
        p = self.p
        return self.tp.lib.tpmlp_kv_append(ref(self.s), ref(self.cache), self.r("q"), self.r("k"), self.r("v"), p["gq"], p["gk"],
                                           p["pos"], p["turns"], p["slot"], self.r("oq"), p["ws"], None)


ENTRIES = ["forward", "backward", "append"]


@pytest.mark.parametrize("entry", ENTRIES)
def test_qk_refuses_shapes_and_null(tp, entry):
    call = lambda c: getattr(c, entry)()
    for bad in BAD_QK:
        assert call(Qk(tp, **bad)) == tp.ERR_INVALID_ARG, bad
    used = {"forward": ("q", "k", "oq", "ok", "gq", "gk", "pos", "turns"),
            "backward": ("q", "k", "dq", "dk", "oq", "ok", "gq", "gk", "pos", "turns", "dgq", "dgk", "ws"),
            "append": ("q", "k", "v", "oq", "gq", "gk", "pos", "turns", "ws", "slot")}[entry]
    for name in used:
        c = Qk(tp)
        if name in c.h:
            c.h[name] = None
            assert call(c) == tp.ERR_INVALID_ARG, name
            c = Qk(tp)
            c.h[name].p = None
        else:
            c.p[name] = None
        assert call(c) == tp.ERR_INVALID_ARG, name
    # pointers that are not on their elements
    for name in used:
        c = Qk(tp)
        if name in c.h:
            c.h[name].p += 1
        else:
            c.p[name] += 1
        assert call(c) == tp.ERR_UNSUPPORTED, name


@pytest.mark.parametrize("entry", ENTRIES)
def test_qk_refuses_rows_that_overlap(tp, entry):
    call = lambda c: getattr(c, entry)()
    for name, n in (("q", 8), ("k", 2), ("oq", 8)):
        for row in (-1, 0, n * 64 - 1, (1 << 40) + 1):
            c = Qk(tp)
            c.h[name].row = row
            assert call(c) == tp.ERR_INVALID_ARG, (name, row)
        for shard in (-1, 0, n // 2 * 64 - 1, (1 << 27) + 1):
            c = Qk(tp, t=2)
            c.h[name].shard = shard
            assert call(c) == tp.ERR_INVALID_ARG, (name, shard)
    # more bytes than an address has
    c = Qk(tp, T=1 << 30)
    c.h["q"].row = 1 << 40
    assert call(c) == tp.ERR_INVALID_ARG


@pytest.mark.parametrize("entry", ENTRIES)
def test_qk_refuses_outputs_over_inputs(tp, entry):
    call = lambda c: getattr(c, entry)()
    pairs = {"forward": [("oq", "k"), ("ok", "q"), ("oq", "ok")],
             "backward": [("oq", "k"), ("ok", "q"), ("oq", "dk"), ("ok", "dq"), ("oq", "ok")],
             "append": [("oq", "k"), ("oq", "v")]}[entry]
    for o, i in pairs:
        for off in (0, 2, 128, 4094):  # (a K is 16 x 128 x 2 bytes)
            c = Qk(tp)
            c.h[o].p = c.h[i].p + off
            assert call(c) == tp.ERR_INVALID_ARG, (o, i, off)
    # in place but moved by an element
    c = Qk(tp)
    c.h["oq"].p = c.h["q"].p + 2
    assert call(c) == tp.ERR_INVALID_ARG
    for name in ("gq", "gk", "pos", "turns") + (("dgq", "dgk") if entry == "backward" else ()) + (("slot",) if entry == "append" else ()):
        c = Qk(tp)
        c.p[name] = c.h["oq"].p + 64
        assert call(c) == tp.ERR_INVALID_ARG, name
    if entry == "backward":
        for a, b in (("dgq", "dgk"), ("dgq", "gk"), ("dgk", "pos")):
            c = Qk(tp)
            c.p[a] = c.p[b]
            assert call(c) == tp.ERR_INVALID_ARG, (a, b)


def test_append_refuses_caches(tp):
    assert Qk(tp, T=0).append() == tp.OK
    for bad in (dict(kv=4), dict(dim=32), dict(dtype=tp.F32), dict(K=None), dict(V=None)):
        c = Qk(tp)
        c.cache = cshape(tp, **bad)
        assert c.append() == tp.ERR_INVALID_ARG, bad
    for name in ("q", "k", "v", "oq"):
        c = Qk(tp)
        c.h[name].p = c.cache.K + 512
        assert c.append() == tp.ERR_INVALID_ARG, name
    for name in ("slot", "pos", "gq"):
        c = Qk(tp)
        c.p[name] = c.cache.V + 64
        assert c.append() == tp.ERR_INVALID_ARG, name
    c = Qk(tp)
    c.cache.K += 1
    assert c.append() in (tp.ERR_INVALID_ARG, tp.ERR_UNSUPPORTED)


# ---- the cache and attention over it ------------------------------------------------------------------

BAD_CACHE = (dict(pages=0), dict(page=0), dict(kv=0), dict(dim=0), dict(dim=63), dict(dim=258), dict(dtype=4), dict(pages=1 << 31),
             dict(pages=1 << 30, page=1 << 11), dict(strides=(-2048, 1024, 64)), dict(strides=(2047, 1024, 64)),
             dict(strides=(2048, 1023, 64)), dict(strides=(2048, 1024, 63)), dict(strides=(0, 1024, 64)), dict(strides=(2048, 0, 64)),
             dict(strides=(2048, 1024, 0)), dict(strides=((1 << 39) + 1, 1024, 64)))


def attend(tp, s, c, p=None, ws=FAKE + (20 << 34)):
    # Q, q_start, kv_len, page_table, tree, O
    p = p or pointers()
    return tp.lib.tpmlp_cache_attn(ref(s) if s else None, ref(c) if c else None, *p, ws, None)


def pointers(**kw):
    names = ("Q", "q_start", "kv_len", "table", "tree", "O")
    return [kw.get(n, None if n == "tree" else FAKE + (2 + i << 34)) for i, n in enumerate(names)]


def test_attention_workspace(tp):
    size = lambda c={}, **k: tp.lib.tpmlp_cache_attn_workspace_bytes(ref(ashape(tp, **k)), ref(cshape(tp, **c)))
    assert size() == size(T=0) == size(batch=1000) == size(c=dict(pages=1 << 20)) > 0  # dim alone
    assert size(c=dict(dim=256)) < 128 << 20
    for bad in (dict(T=-1), dict(batch=-1), dict(batch=(1 << 20) + 1), dict(max_pages=-1), dict(max_pages=1 << 27), dict(heads=0),
                dict(heads=7), dict(T=1 << 28), dict(T=1 << 31, heads=2), dict(algo=7), dict(words=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(scale=3e38)):
        assert size(**bad) == 0, bad
        assert attend(tp, ashape(tp, **bad), cshape(tp)) == tp.ERR_INVALID_ARG, bad
    for bad in BAD_CACHE:
        assert size(c=bad) == 0, bad
        assert attend(tp, ashape(tp), cshape(tp, **bad)) == tp.ERR_INVALID_ARG, bad


def test_attention_refusals(tp):
    s, c = ashape(tp), cshape(tp)
    assert attend(tp, None, c) == tp.ERR_INVALID_ARG and attend(tp, s, None) == tp.ERR_INVALID_ARG
    assert attend(tp, s, c, ws=None) == tp.ERR_INVALID_ARG
    for name in ("Q", "q_start", "kv_len", "table", "O"):
        assert attend(tp, s, c, pointers(**{name: None})) == tp.ERR_INVALID_ARG, name
    assert attend(tp, s, cshape(tp, K=None)) == tp.ERR_INVALID_ARG and attend(tp, s, cshape(tp, V=None)) == tp.ERR_INVALID_ARG
    tree = FAKE + (9 << 34)
    assert attend(tp, s, c, pointers(tree=tree)) == tp.ERR_INVALID_ARG  # without words
    for name, off in (("Q", 8), ("O", 8), ("Q", 2), ("q_start", 2), ("kv_len", 2), ("table", 2)):
        p = pointers()
        p[("Q", "q_start", "kv_len", "table", "tree", "O").index(name)] += off
        assert attend(tp, s, c, p) == tp.ERR_UNSUPPORTED, name
    assert attend(tp, ashape(tp, words=1), c, pointers(tree=tree + 4)) == tp.ERR_UNSUPPORTED
    assert attend(tp, s, c, ws=FAKE + 8) == tp.ERR_UNSUPPORTED
    for dim in (2, 12, 62, 132, 254):
        assert attend(tp, s, cshape(tp, dim=dim)) == tp.ERR_UNSUPPORTED, dim
    o = pointers()[5]
    for name in ("Q", "q_start", "kv_len", "table"):
        assert attend(tp, s, c, pointers(**{name: o + 16})) == tp.ERR_INVALID_ARG, name
    assert attend(tp, ashape(tp, words=1), c, pointers(tree=o + 64)) == tp.ERR_INVALID_ARG
    assert attend(tp, s, cshape(tp, K=o + 64)) == tp.ERR_INVALID_ARG and attend(tp, s, cshape(tp, V=o - 64)) == tp.ERR_INVALID_ARG
    # nothing to do
    for empty in (dict(T=0), dict(batch=0), dict(T=0, batch=0)):
        assert attend(tp, ashape(tp, **empty), c) == tp.OK


def test_caches_of_many_layouts(tp):
    """Any order of pages, heads and tokens whose rows are apart, K and V interleaved too, is valid."""
    size = lambda **k: tp.lib.tpmlp_cache_attn_workspace_bytes(ref(ashape(tp)), ref(cshape(tp, **k)))
    counts = dict(pages=8, kv=2, page=16)
    for order in itertools.permutations(("pages", "kv", "page")):
        stride, at = {}, 64
        for n in order:
            stride[n], at = at, at * counts[n]
        strides = (stride["pages"], stride["kv"], stride["page"])
        assert size(strides=strides) > 0, order
        # K and V in turns: of every row, and of every page
        assert size(strides=tuple(2 * x for x in strides), V=FAKE + 128) > 0
        assert size(strides=tuple(2 * x for x in strides), V=FAKE + 126) == 0
    assert size(strides=(4096, 1024, 64), V=FAKE + 2 * 2048) > 0
    assert size(strides=(4095, 1024, 64), V=FAKE + 2 * 2048) == 0
    assert size(V=FAKE) == 0


def test_contexts(tp):
    import torch
    bad = [lambda: tp.RopeTable(64, layout="pairs", device="cpu"), lambda: tp.RopeTable(64, scaling=("more", 2.0), device="cpu"),
           lambda: tp.RopeTable(64, scaling=("linear",), device="cpu"), lambda: tp.RopeTable(64, scaling=("parts", 2.0), device="cpu"),
           lambda: tp.RopeTable(63, device="cpu"), lambda: tp.QkContext(4, 8, 3, 64, torch.float16, device="cpu"),
           lambda: tp.QkContext(4, 8, 3, 64, torch.bfloat16, t=2, device="cpu"), lambda: tp.QkContext(4, 8, 2, 63, torch.bfloat16, device="cpu"),
           lambda: tp.QkContext(4, 8, 2, 64, torch.bfloat16, tp.RopeTable(128, device="cpu"), device="cpu"),
           lambda: tp.CacheAttnContext(4, 1, 8, 3, 64, torch.bfloat16, device="cpu"),
           lambda: tp.CacheAttnContext(4, 1, 8, 2, 64, torch.float16, device="cpu"),
           lambda: tp.CacheAttnContext(4, 1, 8, 2, 64, torch.bfloat16, scale=float("inf"), device="cpu"),
           lambda: tp.CacheAttnContext(-1, 1, 8, 2, 64, torch.bfloat16, device="cpu"),
           lambda: tp.KvCache(4, 16, 2, 64, torch.bfloat16, device="cpu"), lambda: tp.KvCache(4, 16, 2, 64, torch.float16, device="cpu")]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, RuntimeError)):
            f()
            pytest.fail(str(i))
    ctx = tp.QkContext(4, 8, 2, 64, torch.bfloat16, tp.RopeTable(64, device="cpu"), device="cpu")
    with pytest.raises(ValueError, match="qk_forward"):
        tp.qk_backward(ctx, None, None)
    with pytest.raises(ValueError):  # tensors that are not on a GPU
        tp.qk_forward(ctx, torch.zeros(4, 12 * 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64))
    ctx._saved = ()
    with pytest.raises(ValueError, match="in place"):
        tp.qk_backward(ctx, None, None)


# ---- the shares of the tiles, restated ------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(40))
def test_shares_cover_every_tile_once(seed):
    """Block c takes the tiles [c total / blocks, (c + 1) total / blocks): every tile is in one block, a cut unit's pieces
    are in consecutive blocks, each block begins at most one unit that it does not end, and the block of the last tile g is
    (g + 1) blocks - 1 over total."""
    rng = random.Random(seed)
    units = [rng.choice((1, 1, 2, 5, rng.randint(1, 400))) for _ in range(rng.randint(1, 300))]
    total, blocks = sum(units), min(sum(units), rng.choice((1, 2, 148, 152, 160)))
    bounds = [c * total // blocks for c in range(blocks + 1)]
    assert all(a < b for a, b in zip(bounds, bounds[1:]))
    sizes = [b - a for a, b in zip(bounds, bounds[1:])]
    assert max(sizes) - min(sizes) <= 1
    begin, open_units = 0, [0] * blocks
    for n in units:
        end = begin + n
        of = [c for c in range(blocks) if bounds[c] < end and bounds[c + 1] > begin]
        assert of == list(range(of[0], of[-1] + 1))
        assert of[-1] == (end * blocks - 1) // total
        if len(of) > 1:
            open_units[of[0]] += 1
            # of its pieces only the first begins the unit; the others are the first thing their blocks do
            assert all(bounds[c] > begin and bounds[c] < end for c in of[1:])
        begin = end
    assert max(open_units) <= 1
