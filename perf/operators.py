"""Measured cases of the two operators at the ends of a training step: the
language-model head's loss with its gradient, and the orthogonalised update.

  xent    softmax cross entropy of X W^T over a vocabulary of V rows, without the
          [T, V] logits being kept: loss and log-sum-exp per token ("score"), or the
          loss and the gradients dX and dW ("train")
  ortho   Newton-Schulz orthogonalisation of gradient matrices:
          X = G/(|G| + eps), then steps of  A = X X^T,  X <- a X + (b A + c A^2) X

Where the module's ``own`` is false, ``run`` computes them with elementary torch
operations in 32 bits; where it is true, through the package's entry points.
"""
import math

import torch

own = False

STEPS = 5
COEF = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
IGNORE = -100

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One token scored against the whole vocabulary (the log-likelihood of a
        # decoded token): W is read once, latency and bandwidth count.
        {"name": "score-token", "op": "score", "T": 1, "h": 4096, "V": 32768, "dtype": "bf16", "ignored": 0.0, "weighted": False},
        # A short prompt scored, odd token count and vocabulary.
        {"name": "score-prompt", "op": "score", "T": 333, "h": 2048, "V": 50021, "dtype": "bf16", "ignored": 0.1, "weighted": False},
        # Evaluation of a whole batch: the h4096 workload's 8192 tokens.
        {"name": "score-h4096", "op": "score", "T": 8192, "h": 4096, "V": 65536, "dtype": "bf16", "ignored": 0.0, "weighted": False},
        # The fp32 workload's tokens and hidden size with a small vocabulary.
        {"name": "train-tiny-f32", "op": "train", "T": 128, "h": 256, "V": 1009, "dtype": "f32", "ignored": 0.2, "weighted": True},
        # Fine-tuning on a ragged batch: prompt tokens ignored, the rest weighted.
        {"name": "train-ragged", "op": "train", "T": 1001, "h": 1000, "V": 30011, "dtype": "bf16", "ignored": 0.3, "weighted": True},
        # The h2048 workload's training step.
        {"name": "train-h2048", "op": "train", "T": 2048, "h": 2048, "V": 32768, "dtype": "bf16", "ignored": 0.0, "weighted": False},
        # The h8192 workload's training step (the largest case).
        {"name": "train-h8192", "op": "train", "T": 4096, "h": 8192, "V": 51200, "dtype": "bf16", "ignored": 0.0, "weighted": False},
        # dA of the smallest workload: every product is tiny, launches count.
        {"name": "ortho-tiny", "op": "ortho", "batch": 1, "rows": 256, "cols": 1024, "dtype": "bf16", "tokens": 128},
        # fp32 gradients of odd-sized matrices, several at once.
        {"name": "ortho-odd-f32", "op": "ortho", "batch": 6, "rows": 515, "cols": 1003, "dtype": "f32", "tokens": 2048},
        # The row blocks of the attention's output projection, one per head.
        {"name": "ortho-heads", "op": "ortho", "batch": 32, "rows": 128, "cols": 4096, "dtype": "bf16", "tokens": 8192},
        # dB of the h2048 workload for four layers: tall matrices.
        {"name": "ortho-h2048-x4", "op": "ortho", "batch": 4, "rows": 8192, "cols": 2048, "dtype": "bf16", "tokens": 2048},
        # dA of the h4096 workload.
        {"name": "ortho-h4096", "op": "ortho", "batch": 1, "rows": 4096, "cols": 16384, "dtype": "bf16", "tokens": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("score", "train", "ortho"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "ortho":
        while True:
            c = {"op": op, "batch": _log(rng, 1, 32), "rows": _log(rng, 16, 8192), "cols": _log(rng, 16, 16384),
                 "dtype": dtype, "tokens": _log(rng, 128, 8192)}
            if c["batch"] * c["rows"] * c["cols"] <= 1 << 26 and work(c)["flops"] <= 3e12:
                return c
    while True:
        f32 = dtype == "f32"
        c = {"op": op, "T": _log(rng, 1, 512 if f32 else 8192), "h": 8 * _log(rng, 4, 128 if f32 else 1024),
             "V": _log(rng, 64, 16384 if f32 else 65536), "dtype": dtype, "ignored": rng.choice((0.0, 0.1, 0.5)),
             "weighted": rng.random() < 0.5}
        if c["T"] * c["h"] * c["V"] <= (1 << 31 if f32 else 1 << 39):
            return c


def _xent_inputs(case, seed):
    """X[T,h], W[V,h], the targets (frequent tokens first, some ignored) and dloss[T].

    X is normalised activations that lean towards the target's row of W by
    different amounts, so that the target's probability runs from that of a
    guess to that of a fair prediction."""
    T, h, V, dt = case["T"], case["h"], case["V"], _DT[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    W = (0.02 * torch.randn(V, h, generator=g, device="cuda")).to(dt)
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    target = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    lean = 5.0 * torch.rand(T, 1, generator=g, device="cuda") / (0.0004 * h)
    X = torch.randn(T, h, generator=g, device="cuda")
    X = (X + lean.clamp_(max=20.0) * W[target].float()).to(dt)
    out = torch.rand(T, generator=g, device="cuda") < case["ignored"]
    out[0] = False
    target = torch.where(out, IGNORE, target)
    w = 2.0 * torch.rand(T, generator=g, device="cuda") if case["weighted"] else torch.ones(T, device="cuda")
    dloss = w / float((~out).sum())
    return X, W, target, dloss


def _ortho_inputs(case, seed):
    """Gradients as a backward pass leaves them: G = U^T D over `tokens` tokens with
    channels of different scales and a common mean, at a gradient's magnitude."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n, r, c, t = case["batch"], case["rows"], case["cols"], case["tokens"]
    U = torch.randn(n, t, r, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(n, 1, r, generator=g, device="cuda"))
    D = torch.randn(n, t, c, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(n, 1, c, generator=g, device="cuda"))
    # half-precision products are exact enough for an input that is random anyway
    return (torch.bmm((U + 0.2).half().transpose(1, 2), D.half()).float() * (1e-4 / t)).to(_DT[case["dtype"]])


def prepare(case, seed):
    if case["op"] == "ortho":
        s = {"case": case, "G": _ortho_inputs(case, seed)}
        if own:
            from tensor_transformer_mlp_tma_gb300 import tpmlp
            s["ctx"] = tpmlp.OrthoContext(case["rows"], case["cols"], case["batch"], _DT[case["dtype"]], steps=STEPS)
        return s
    X, W, target, dloss = _xent_inputs(case, seed)
    s = {"case": case, "X": X, "W": W, "target": target, "dloss": dloss}
    if own:
        from tensor_transformer_mlp_tma_gb300 import tpmlp
        s["ctx"] = tpmlp.XentContext(case["T"], case["h"], case["V"], _DT[case["dtype"]], ignore_index=IGNORE)
    return s


def _plain_xent(s, train):
    X, W, target = s["X"].float(), s["W"].float(), s["target"]
    valid = target != IGNORE
    at = torch.where(valid, target, 0)[:, None]
    S = X @ W.t()
    m = S.amax(1, keepdim=True)
    z = S.gather(1, at)
    S.sub_(m).exp_()
    n = S.sum(1, keepdim=True)
    loss = torch.where(valid, ((m - z) + n.log())[:, 0], 0.0)
    if not train:
        return {"loss": loss, "lse": (m + n.log())[:, 0]}
    g = torch.where(valid, s["dloss"], 0.0)[:, None]
    S.mul_(g / n)
    S.scatter_add_(1, at, -g)
    return {"loss": loss, "dX": (S @ W).to(s["X"].dtype), "dW": (S.t() @ X).to(s["W"].dtype)}


def _step(X):
    a, b, c = COEF
    A = torch.bmm(X, X.transpose(1, 2))
    B = torch.baddbmm(A, A, A, beta=b, alpha=c)
    return torch.baddbmm(X, B, X, beta=a)


def _plain_ortho(G, wide):
    X = G.float() if wide else G.float().transpose(1, 2)
    big = X.abs().amax((1, 2), keepdim=True).clamp_min(1e-30)
    norm = (X / big).square().sum((1, 2), keepdim=True).sqrt() * big
    X = X / (norm + EPS)
    for _ in range(STEPS):
        X = _step(X)
    return (X if wide else X.transpose(1, 2)).to(torch.bfloat16).contiguous()


def run(s):
    case = s["case"]
    if own:
        from tensor_transformer_mlp_tma_gb300 import tpmlp
        if case["op"] == "ortho":
            return tpmlp.orthogonalize(s["ctx"], s["G"])
        loss = tpmlp.xent_forward(s["ctx"], s["X"], s["W"], s["target"])
        if case["op"] == "score":
            return {"loss": loss, "lse": s["ctx"].lse}
        grads = tpmlp.xent_backward(s["ctx"], s["dloss"])
        return {"loss": loss, "dX": grads["dX"], "dW": grads["dW"]}
    if case["op"] == "ortho":
        return _plain_ortho(s["G"], case["rows"] <= case["cols"])
    return _plain_xent(s, case["op"] == "train")


def work(case):
    """Bytes: inputs read once, outputs written once.  FLOPs: xent 2ThV for the
    logits and 4ThV for dX and dW; ortho per step, with p <= q the two sizes, the
    lower triangles of the symmetric A (p^2 q) and A^2 (p^3) and the product 2 p^2 q."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "ortho":
        n, p, q = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        return {"bytes": n * p * q * (e + 2), "flops": STEPS * n * (3.0 * p * p * q + 1.0 * p * p * p)}
    T, h, V = case["T"], case["h"], case["V"]
    inputs = e * (T * h + V * h) + 8 * T
    if case["op"] == "score":
        return {"bytes": inputs + 8 * T, "flops": 2.0 * T * h * V}
    return {"bytes": inputs + 4 * T + 4 * T + e * (T * h + V * h), "flops": 6.0 * T * h * V}


def exact(case, seed):
    if work(case)["flops"] > 1.4e13:
        return None
    if case["op"] == "ortho":
        a, b, c = COEF
        G = _ortho_inputs(case, seed).double()
        out = torch.empty_like(G)
        for i in range(G.shape[0]):
            X = G[i] if G.shape[1] <= G.shape[2] else G[i].t()
            X = X / (torch.linalg.vector_norm(X) + EPS)
            one = torch.eye(X.shape[0], dtype=torch.float64, device=X.device)
            for _ in range(STEPS):
                A = X @ X.t()
                X = (a * one + A @ (b * one + c * A)) @ X
            out[i] = X if G.shape[1] <= G.shape[2] else X.t()
        return out
    X, W, target, dloss = _xent_inputs(case, seed)
    X, W, dloss = X.double(), W.double(), dloss.double()
    T, train = X.shape[0], case["op"] == "train"
    loss, lse, dX = (torch.zeros(n, dtype=torch.float64, device="cuda") for n in ((T,), (T,), X.shape))
    dW = torch.zeros_like(W) if train else None
    for i in range(0, T, 1024):
        r = slice(i, min(i + 1024, T))
        S = X[r] @ W.t()
        lse[r] = torch.logsumexp(S, 1)
        k = (target[r] != IGNORE).nonzero()[:, 0]
        loss[i + k] = lse[i + k] - S[k, target[i + k]]
        if train:
            P = torch.exp(S - lse[r, None])
            P[k, target[i + k]] -= 1.0
            g = torch.zeros(P.shape[0], dtype=torch.float64, device="cuda")
            g[k] = dloss[i + k]
            P *= g[:, None]
            dX[r] = P @ W
            dW += P.t() @ X[r]
    return {"loss": loss, "dX": dX, "dW": dW} if train else {"loss": loss, "lse": lse}
