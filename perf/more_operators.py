"""Measured cases of positions and the key-value cache of the attention block.

  qk      per-head norms of queries and keys and the position rotation in one pass over the
          projected QKV; a training step returns the gradients too
  append  keys (normed, rotated) and values of new tokens into a paged cache, the new queries
          normed and rotated beside them
  attend  attention of new tokens over the paged cache: one token per sequence, a prompt's
          chunk (causal), or a tree of drafted tokens

    y = g x / sqrt(mean(x^2) + eps)                     (norm, per head, gains g [d])
    (u, v) -> a (u cos f - v sin f, u sin f + v cos f)  (rotation by f = position * theta_i)
    O = softmax(scale Q K^T over the visible keys) V

Where the module's ``own`` is false, ``run`` computes them with elementary torch operations in
32 bits (angles in 64); where it is true, through the package's entry points.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0
CONTEXT, LOW, HIGH = 2048, 1.0, 32.0  # of the scaling by parts
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _qk(name, T, heads, kv, d, t, rot, layout, norm, dtype, train, scaling="", factor=1.0, far=0):
    return {"name": name, "op": "qk", "T": T, "heads": heads, "kv": kv, "d": d, "t": t, "rot": rot, "layout": layout,
            "norm": norm, "dtype": dtype, "train": train, "scaling": scaling, "factor": factor, "far": far}


def _append(name, batch, new_lo, new_hi, heads, kv, d, page, rot, layout, norm, dtype, skip, far):
    return {"name": name, "op": "append", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "heads": heads, "kv": kv,
            "d": d, "page": page, "rot": rot, "layout": layout, "norm": norm, "dtype": dtype, "skip": skip, "far": far}


def _attend(name, batch, lo, hi, new_lo, new_hi, tree, heads, kv, d, page, dtype):
    return {"name": name, "op": "attend", "batch": batch, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi,
            "tree": tree, "heads": heads, "kv": kv, "d": d, "page": page, "dtype": dtype}


def listed():
    return [
        # The fp32 workload's 128 tokens of width 256: a training step where launches count.
        _qk("qk-tiny-f32", 128, 4, 4, 64, 1, 64, "half", True, "f32", True),
        # A training step of the h4096 attention workload: 4 sequences of 2048, 32 heads, 8 shards.
        _qk("qk-h4096-train", 8192, 32, 32, 128, 8, 128, "half", True, "bf16", True),
        # The h8192 workload's prompt, scored: rotation alone, neighbouring pairs, half of each head.
        _qk("qk-h8192-rotate", 4096, 64, 64, 128, 8, 64, "interleaved", False, "bf16", False),
        # Odd sizes, shared key heads, far positions of a model stretched to a longer context.
        _qk("qk-odd-far", 1001, 6, 2, 80, 2, 48, "half", True, "bf16", True, "parts", 8.0, 1 << 20),
        # One decoded token of one sequence: latency.
        _append("append-token", 1, 1, 1, 32, 32, 128, 16, 128, "half", True, "bf16", 0.0, 2000),
        # A batch of drafts, 1 to 8 tokens each, a tenth of them padding.
        _append("append-drafts", 61, 1, 8, 32, 8, 128, 16, 96, "interleaved", False, "bf16", 0.1, 100000),
        # Prompts of 4 sequences, 8192 tokens at most.
        _append("append-prompt", 4, 1500, 2048, 64, 8, 128, 64, 128, "half", True, "bf16", 0.0, 0),
        # One token of one sequence of the h4096 workload's length, every head with its own keys.
        _attend("attend-token", 1, 2047, 2047, 1, 1, False, 32, 32, 128, 16, "bf16"),
        # A batch in decoding, lengths from short to 8192, shared key heads.
        _attend("attend-batch", 64, 100, 8192, 1, 1, False, 32, 8, 128, 16, "bf16"),
        # Trees of up to 64 drafted tokens on 16 sequences.
        _attend("attend-tree", 16, 500, 4096, 17, 64, True, 32, 8, 128, 16, "bf16"),
        # One long sequence: 8 drafted tokens over 131072 cached ones.
        _attend("attend-long", 1, 131064, 131064, 8, 8, True, 64, 8, 128, 64, "bf16"),
        # Chunks of 4 prompts of the h8192 workload over what is cached of them (the largest case).
        _attend("attend-chunk", 4, 3000, 8192, 300, 512, False, 64, 8, 128, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice((1, 2, 3, 4, 8, 8, 16, 32))
    return kv * rng.choice((1, 1, 2, 4, 8) if kv <= 8 else (1, 2)), kv


def draw(rng):
    op = rng.choice(("qk", "append", "attend", "attend"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    layout, norm = rng.choice(("half", "interleaved")), rng.random() < 0.6
    while True:
        heads, kv = _heads(rng)
        d = rng.choice((32, 64, 64, 80, 96, 128, 128, 128, 192, 256))
        rot = rng.choice((d, d, d // 2, 16))
        page = rng.choice((8, 16, 16, 32, 48, 64, 128))
        if op == "qk":
            t = rng.choice([n for n in (1, 2, 4, 8) if kv % n == 0])
            c = _qk("", _log(rng, 1, 8192), heads, kv, d, t, rot, layout, norm, dtype, rng.random() < 0.6,
                    *rng.choice((("", 1.0), ("linear", 4.0), ("parts", 8.0))), rng.choice((0, 10000, 1 << 20)))
            fits = c["T"] * (heads + kv) * d <= 8192 * 64 * 128
        elif op == "append":
            lo = _log(rng, 1, 512)
            c = _append("", _log(rng, 1, 128), lo, _log(rng, lo, 2 * lo), heads, kv, d, page, rot, layout, norm, dtype,
                        rng.choice((0.0, 0.1)), rng.choice((0, 3000, 200000)))
            fits = c["batch"] * c["new_hi"] * (heads + 2 * kv) * d <= 8192 * 80 * 128
        else:
            f32 = dtype == "f32"
            lo, new = _log(rng, 1, 2000 if f32 else 32768), _log(rng, 1, 64 if f32 else 256)
            c = _attend("", _log(rng, 1, 64), lo, _log(rng, lo, 4 * lo), rng.randint(1, new), new, rng.random() < 0.5,
                        heads, kv, d, page, dtype)
            w, most = work(c), work(listed()[-1])
            padded = c["batch"] * (c["hi"] + new) * max(kv * d, heads * new / 4)  # of the plain form
            fits = w["bytes"] <= 1 << 30 and w["flops"] <= most["flops"] / (8 if f32 else 1) and padded <= 1 << 29
        if fits:
            del c["name"]
            return c


def _lengths(case):
    """(cached tokens, new tokens) of each sequence, the same for every seed."""
    rng = random.Random("%(batch)d %(new_lo)d %(new_hi)d" % case + str(case.get("hi", case.get("far"))))
    lo, hi = (case["lo"], case["hi"]) if case["op"] == "attend" else (case["far"] // 2, case["far"])
    return [(rng.randint(lo, hi), rng.randint(case["new_lo"], case["new_hi"])) for _ in range(case["batch"])]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tokens(case):
    return case["T"] if case["op"] == "qk" else sum(n for _, n in _lengths(case))


def _projected(case, g):
    """QKV as a projection leaves it: channels of different scales, and the gains."""
    T, heads, kv, d, dt = _tokens(case), case["heads"], case["kv"], case["d"], _DT[case["dtype"]]
    scale = torch.exp(0.4 * torch.randn((heads + 2 * kv) * d, generator=g, device="cuda"))
    QKV = (scale * torch.randn(T, (heads + 2 * kv) * d, generator=g, device="cuda")).to(dt)
    gains = [(1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if case["norm"] else None for _ in "qk"]
    return QKV, gains[0], gains[1]


def _qk_inputs(case, seed):
    g = _generator(seed)
    QKV, gq, gk = _projected(case, g)
    T = case["T"]
    s = {"QKV": QKV, "gq": gq, "gk": gk}
    # sequences of 2048, each at an offset of its own
    offset = torch.randint(0, case["far"] + 1, ((T + 2047) // 2048,), generator=g, device="cuda")
    at = torch.arange(T, device="cuda")
    s["position"] = at % 2048 + offset[at // 2048]
    if case["train"]:
        for name, n in (("dQ", case["heads"]), ("dK", case["kv"])):
            s[name] = (0.01 * torch.randn(T, n, case["d"], generator=g, device="cuda")).to(QKV.dtype)
    return s


def _pages(counts, spare, g):
    """Page numbers for sequences that need `counts` pages each, in no order, and how many there are."""
    n = sum(counts) + spare
    order = torch.randperm(n, generator=g, device="cuda")
    table = torch.zeros(len(counts), max(max(counts), 1), dtype=torch.int64)
    of = [(b, i) for b, c in enumerate(counts) for i in range(c)]
    if of:
        b, i = torch.tensor(of).t()
        table[b, i] = order.cpu()[:len(of)]
    return table.cuda(), n


def _append_inputs(case, seed):
    g = _generator(seed)
    QKV, gq, gk = _projected(case, g)
    page, lens = case["page"], _lengths(case)
    # the pages that the new tokens reach
    table, pages = _pages([(c + n - 1) // page - c // page + 1 for c, n in lens], 4, g)
    seq = torch.tensor([b for b, (_, n) in enumerate(lens) for _ in range(n)], device="cuda")
    position = torch.tensor([c + i for c, n in lens for i in range(n)], device="cuda")
    first = torch.tensor([c // page for c, _ in lens], device="cuda")
    slot = table[seq, position // page - first[seq]] * page + position % page
    slot = torch.where(torch.rand(len(seq), generator=g, device="cuda") < case["skip"], -1, slot)
    cache = torch.randn(2, pages, case["kv"], page, case["d"], generator=g, device="cuda").to(QKV.dtype)
    return {"QKV": QKV, "gq": gq, "gk": gk, "position": position, "slot": slot, "cache": cache}


def _attend_inputs(case, seed):
    """Rotated queries and keys: a few keys that every query looks at, and queries that lean towards
    some key, so that the weights run from even to one key's alone."""
    g = _generator(seed)
    heads, kv, d, page, dt = case["heads"], case["kv"], case["d"], case["page"], _DT[case["dtype"]]
    lens = _lengths(case)
    table, pages = _pages([(c + n + page - 1) // page for c, n in lens], 8, g)
    K, V = (torch.randn(pages, kv, page, d, generator=g, device="cuda") for _ in "kv")
    K += torch.where(torch.rand(pages, kv, page, 1, generator=g, device="cuda") < 0.01, 0.5, 0.1)
    T = sum(n for _, n in lens)
    Q = torch.randn(T, heads, d, generator=g, device="cuda")
    near = torch.randint(0, pages * page, (T, kv), generator=g, device="cuda")
    key = K[near // page, torch.arange(kv, device="cuda"), near % page]
    Q += 0.5 * torch.rand(T, 1, 1, generator=g, device="cuda") * key.repeat_interleave(heads // kv, 1)
    s = {"Q": Q.to(dt), "K": K.to(dt), "V": V.to(dt), "table": table.int()}
    s["kv_len"] = torch.tensor([c + n for c, n in lens], dtype=torch.int32, device="cuda")
    starts = [sum(n for _, n in lens[:b]) for b in range(len(lens) + 1)]
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["tree"] = None
    if case["tree"]:
        # token i of a draft continues an earlier one or the text itself; bit j: token j is i or above it
        words = (max(n for _, n in lens) + 63) // 64
        rng = random.Random(seed)
        masks = []
        for _, n in lens:
            of = []
            for i in range(n):
                above = rng.randint(max(-1, i - 8), i - 1)
                of.append((of[above] if above >= 0 else 0) | 1 << i)
            masks += of
        signed = [[(m >> 64 * w & (1 << 64) - 1) - (1 << 64 if m >> 64 * w + 63 & 1 else 0) for w in range(words)] for m in masks]
        s["tree"] = torch.tensor(signed, dtype=torch.int64, device="cuda")
    return s


def prepare(case, seed):
    s = {"qk": _qk_inputs, "append": _append_inputs, "attend": _attend_inputs}[case["op"]](case, seed)
    s["case"] = case
    if case["op"] == "attend":
        lens = _lengths(case)
        # where each new token goes in a batch padded to the longest draft
        s["seq"] = torch.tensor([b for b, (_, n) in enumerate(lens) for _ in range(n)], device="cuda")
        s["at"] = torch.tensor([i for _, n in lens for i in range(n)], device="cuda")
        s["widest"] = max(n for _, n in lens)
    else:
        s["theta"] = torch.tensor(_theta(case), dtype=torch.float64, device="cuda")
    if own:
        from tensor_transformer_mlp_tma_gb300 import tpmlp
        heads, kv, d, dt = case["heads"], case["kv"], case["d"], _DT[case["dtype"]]
        if case["op"] == "attend":
            s["cache"] = tpmlp.KvCache.of(s["K"], s["V"])
            s["ctx"] = tpmlp.CacheAttnContext(s["Q"].shape[0], case["batch"], heads, kv, d, dt)
        else:
            scaling = {"": None, "linear": ("linear", case.get("factor")),
                       "parts": ("parts", case.get("factor"), CONTEXT, LOW, HIGH)}[case.get("scaling", "")]
            rope = tpmlp.RopeTable(case["rot"], BASE, case["layout"], scaling)
            s["ctx"] = tpmlp.QkContext(_tokens(case), heads, kv, d, dt, rope, norm=case["norm"], eps=EPS, t=case.get("t", 1))
            if case["op"] == "append":
                s["kv"] = tpmlp.KvCache.of(s["cache"][0], s["cache"][1])
    return s


def _theta(case):
    """The angle per position of each pair, stretched where the case says so."""
    theta = [BASE ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]
    scaling, factor = case.get("scaling", ""), case.get("factor", 1.0)
    if scaling == "linear":
        return [f / factor for f in theta]
    if scaling == "parts":
        keep = [min(1.0, max(0.0, (CONTEXT * f / (2 * math.pi) - LOW) / (HIGH - LOW))) for f in theta]
        return [f * (k + (1.0 - k) / factor) for f, k in zip(theta, keep)]
    return theta


def _split(case, QKV):
    """Q [T, heads, d], K and V [T, kv, d] out of the projection's shard-major columns."""
    t, d = case.get("t", 1), case["d"]
    n, m = case["heads"] // t, case["kv"] // t
    x = QKV.view(-1, t, n + 2 * m, d)
    return x[:, :, :n].reshape(-1, n * t, d), x[:, :, n:n + m].reshape(-1, m * t, d), x[:, :, n + m:].reshape(-1, m * t, d)


def _pairs(case, x):
    """The two members of every pair, and the rest of the head."""
    rot = case["rot"]
    if case["layout"] == "half":
        return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
    return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]


def _joined(case, u, v, rest):
    rotated = torch.cat((u, v), -1) if case["layout"] == "half" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((rotated, rest), -1)


def _rotated(case, x, cos, sin):
    u, v, rest = _pairs(case, x)
    return _joined(case, u * cos - v * sin, u * sin + v * cos, rest)


def _angles(s):
    f = s["position"].double()[:, None] * s["theta"]
    return f.cos().float()[:, None], f.sin().float()[:, None]


def _plain_norm(x, gain):
    if gain is None:
        return x, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r * gain.float(), r


def _plain_back(case, x, r, gain, dy, cos, sin):
    """Gradients of one of Q and K: x before the norm, dy of what the rotation returned."""
    dy = _rotated(case, dy.float(), cos, -sin)
    if gain is None:
        return dy, None
    xhat = x * r
    dg = (dy * xhat).sum((0, 1))
    g = dy * gain.float()
    return r * (g - xhat * (g * xhat).mean(-1, keepdim=True)), dg


def _plain_qk(s):
    case = s["case"]
    dt = s["QKV"].dtype
    Q, K, _ = (x.float() for x in _split(case, s["QKV"]))
    cos, sin = _angles(s)
    Qn, rq = _plain_norm(Q, s["gq"])
    Kn, rk = _plain_norm(K, s["gk"])
    out = {"Q": _rotated(case, Qn, cos, sin).to(dt), "K": _rotated(case, Kn, cos, sin).to(dt)}
    if case["train"]:
        dQ, dgq = _plain_back(case, Q, rq, s["gq"], s["dQ"], cos, sin)
        dK, dgk = _plain_back(case, K, rk, s["gk"], s["dK"], cos, sin)
        out.update(dQ=dQ.to(dt), dK=dK.to(dt))
        if case["norm"]:
            out.update(dgain_q=dgq.to(dt), dgain_k=dgk.to(dt))
    return out


def _plain_append(s):
    case, cache, slot = s["case"], s["cache"], s["slot"]
    Q, K, V = _split(case, s["QKV"])
    cos, sin = _angles(s)
    Q = _rotated(case, _plain_norm(Q.float(), s["gq"])[0], cos, sin).to(cache.dtype)
    K = _rotated(case, _plain_norm(K.float(), s["gk"])[0], cos, sin).to(cache.dtype)
    keep = (slot >= 0).nonzero()[:, 0]
    page, at = slot[keep] // case["page"], slot[keep] % case["page"]
    cache[0][page, :, at] = K[keep]
    cache[1][page, :, at] = V[keep]
    return {"Q": Q, "K": cache[0], "V": cache[1]}


def _visible(s, keys):
    """[batch, widest, keys]: which keys each token of the padded batch sees."""
    case, n = s["case"], s["widest"]
    length = s["kv_len"].long()[:, None, None]
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()[:, None, None]
    key = torch.arange(keys, device="cuda")[None, None]
    of = key - (length - new)  # number of the drafted token that the key belongs to
    if s["tree"] is None:
        return of <= torch.arange(n, device="cuda")[None, :, None]
    mask = torch.zeros(case["batch"], n, s["tree"].shape[1], dtype=torch.int64, device="cuda")
    mask[s["seq"], s["at"]] = s["tree"]
    bit = of.clamp(0, 64 * mask.shape[2] - 1)
    word = mask.gather(2, (bit // 64).expand(-1, n, -1))
    return (of < 0) | ((word >> bit % 64 & 1).bool() & (of < new))


def _plain_attend(s):
    case, Q = s["case"], s["Q"]
    B, n, heads, kv, d = case["batch"], s["widest"], case["heads"], case["kv"], case["d"]
    q = torch.zeros(B, n, heads, d, device="cuda")
    q[s["seq"], s["at"]] = Q.float()
    q = q.view(B, n, kv, heads // kv, d).permute(0, 2, 1, 3, 4).reshape(B, kv, -1, d)
    K, V = (x[s["table"].long()].float().transpose(1, 2).reshape(B, kv, -1, d) for x in (s["K"], s["V"]))
    S = (q @ K.transpose(2, 3)).view(B, kv, n, heads // kv, -1) / math.sqrt(d)
    S = S.masked_fill_(~_visible(s, S.shape[-1])[:, None, :, None], -math.inf)
    top = S.amax(-1, keepdim=True).clamp_min(-1e30)
    P = S.sub_(top).exp_()
    total = P.sum(-1, keepdim=True)
    O = (P.view(B, kv, -1, P.shape[-1]) @ V).view(B, kv, n, heads // kv, d) / total.clamp_min(1e-30)
    O = O.permute(0, 2, 1, 3, 4).reshape(B, n, heads, d)
    return O[s["seq"], s["at"]].to(Q.dtype)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"qk": _plain_qk, "append": _plain_append, "attend": _plain_attend}[op](s)
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    case, ctx = s["case"], s["ctx"]
    if op == "attend":
        return tpmlp.cache_attention(ctx, s["cache"], s["Q"], s["q_start"], s["kv_len"], s["table"], s["tree"])
    if op == "append":
        Q = tpmlp.kv_append(ctx, s["kv"], s["QKV"], s["position"], s["slot"], s["gq"], s["gk"])
        return {"Q": Q, "K": s["cache"][0], "V": s["cache"][1]}
    Q, K = tpmlp.qk_forward(ctx, s["QKV"], s["position"], s["gq"], s["gk"])
    out = {"Q": Q, "K": K}
    if case["train"]:
        grads = tpmlp.qk_backward(ctx, s["dQ"], s["dK"])
        out.update(dQ=grads["dQ"], dK=grads["dK"])
        if case["norm"]:
            out.update(dgain_q=grads["dgain_q"], dgain_k=grads["dgain_k"])
    return out


def work(case):
    """Bytes: inputs read once, outputs written once (of the cache, what is read or written of it).
    FLOPs: 4 per visible key, head and component; 8 to 20 per component of a norm and rotation."""
    e = 2 if case["dtype"] == "bf16" else 4
    T, heads, kv, d = _tokens(case), case["heads"], case["kv"], case["d"]
    if case["op"] == "qk":
        n = T * (heads + kv) * d
        return {"bytes": (5 if case["train"] else 2) * n * e + 8 * T, "flops": (28.0 if case["train"] else 8.0) * n}
    if case["op"] == "append":
        return {"bytes": 2 * T * (heads + 2 * kv) * d * e + 16 * T, "flops": 8.0 * T * (heads + kv) * d}
    lens = _lengths(case)
    keys = sum(c + n for c, n in lens)
    seen = sum(n * c + n * (n + 1) / 2 for c, n in lens)
    return {"bytes": 2 * keys * kv * d * e + 2 * T * heads * d * e, "flops": 4.0 * seen * heads * d}


def _exact_qk(case, QKV, gains, position):
    """Q, K and V, normed and rotated (as complex numbers), and Q and K before."""
    t, d, rot = case.get("t", 1), case["d"], case["rot"]
    a, b = case["heads"] // t * d, case["kv"] // t * d
    shards = QKV.double().chunk(t, 1)
    raw = [torch.cat([s[:, i:j] for s in shards], 1).view(len(QKV), -1, d) for i, j in ((0, a), (a, a + b), (a + b, a + 2 * b))]
    out = []
    turn = torch.polar(torch.ones(len(QKV), rot // 2, dtype=torch.float64, device="cuda"),
                       position.double()[:, None] * torch.tensor(_theta(case), dtype=torch.float64, device="cuda"))
    for i, (x, gain) in enumerate(zip(raw[:2], gains)):
        x.requires_grad_(True)
        y = x if gain is None else gain * x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS)
        if case["layout"] == "half":
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn[:, None]
            y = torch.cat((z.real, z.imag, y[..., rot:]), -1)
        else:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn[:, None]
            y = torch.cat((torch.view_as_real(z).flatten(-2), y[..., rot:]), -1)
        out.append(y)
    return out + [raw[2]], raw


def exact(case, seed):
    if case["op"] == "qk":
        s = _qk_inputs(case, seed)
        gains = [None if g is None else g.double().requires_grad_(True) for g in (s["gq"], s["gk"])]
        out, raw = _exact_qk(case, s["QKV"], gains, s["position"])
        r = {"Q": out[0].detach(), "K": out[1].detach()}
        if case["train"]:
            ((out[0] * s["dQ"].double()).sum() + (out[1] * s["dK"].double()).sum()).backward()
            r.update(dQ=raw[0].grad, dK=raw[1].grad)
            if case["norm"]:
                r.update(dgain_q=gains[0].grad, dgain_k=gains[1].grad)
        return r
    if case["op"] == "append":
        s = _append_inputs(case, seed)
        gains = [None if g is None else g.double() for g in (s["gq"], s["gk"])]
        out, _ = _exact_qk(case, s["QKV"], gains, s["position"])
        cache = s["cache"].double().transpose(2, 3).contiguous()
        pool = cache.view(2, -1, case["kv"], case["d"])
        kept = s["slot"] >= 0
        pool[0, s["slot"][kept]] = out[1].detach()[kept]
        pool[1, s["slot"][kept]] = out[2].detach()[kept]
        cache = cache.transpose(2, 3).contiguous()
        return {"Q": out[0].detach(), "K": cache[0], "V": cache[1]}
    if work(case)["flops"] > 2e12:
        return None
    s = _attend_inputs(case, seed)
    heads, kv, d = case["heads"], case["kv"], case["d"]
    out = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    q0 = 0
    for b, (cached, n) in enumerate(_lengths(case)):
        slots = torch.arange(cached + n, device="cuda")
        page = s["table"][b].long()[slots // case["page"]]
        K, V = (x[page, :, slots % case["page"]].double() for x in (s["K"], s["V"]))
        seen = torch.ones(n, cached + n, dtype=torch.bool, device="cuda")
        if s["tree"] is None:
            seen[:, cached:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            j = torch.arange(n, device="cuda")
            seen[:, cached:] = (s["tree"][q0:q0 + n][:, j // 64] >> (j % 64) & 1).bool()
        for h in range(heads):
            S = (s["Q"][q0:q0 + n, h].double() @ K[:, h * kv // heads].t() / math.sqrt(d)).masked_fill(~seen, -math.inf)
            out[q0:q0 + n, h] = torch.softmax(S, 1) @ V[:, h * kv // heads]
        q0 += n
    return out
