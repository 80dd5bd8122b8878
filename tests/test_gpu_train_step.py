"""A training step over the library's parts as they are used together: the MLP block forward,
the vocabulary cross entropy on its output, its gradient as the block's dZ, the block
backward, and the orthogonalised update of the weight gradients; eagerly, captured into a
graph, and two steps at once on two streams.

Each stage is compared with 64 bits from the stage's own inputs, with the tolerances of that
stage's tests (max error over max for the block's outputs, as in the parity tests)."""
import pytest
import torch

from tensor_transformer_mlp_tma_gb300 import inputs

pytestmark = pytest.mark.gpu

T, H, F, V, SHARDS = 384, 256, 1024, 3001, 4


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


class Step:
    def __init__(self, tp, seed):
        d = inputs.make(T, H, F, "bf16", seed, {"A": 0.05, "B": 0.05, "a": 0.1, "b": 0.1})
        self.d = {k: v.cuda() for k, v in d.items()}
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        self.W = (torch.randn(V, H, generator=g) * 0.1).bfloat16().cuda()
        self.y = torch.randint(0, V, (T,), generator=g).cuda()
        self.y[::7] = -100
        self.dloss = torch.full((T,), 1.0 / T, device="cuda")
        self.block = tp.Context(T, H, F, SHARDS, torch.bfloat16)
        self.head = tp.XentContext(T, H, V, torch.bfloat16, piece=1024)
        self.update = {"dA": tp.OrthoContext(H, F), "dB": tp.OrthoContext(F, H)}
        self.tp = tp
        e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")
        self.out = {"Z": e(T, H), "loss": e(T, dt=torch.float32), "dZ": e(T, H), "dW": e(V, H), "dX": e(T, H),
                    "dA": e(H, F), "da": e(F), "dB": e(F, H), "db": e(H), "OA": e(H, F), "OB": e(F, H)}

    def run(self):
        tp, d, o = self.tp, self.d, self.out
        tp.forward(self.block, d["X"], d["A"], d["a"], d["B"], d["b"], o["Z"])
        tp.xent_forward(self.head, o["Z"], self.W, self.y, o["loss"])
        tp.xent_backward(self.head, self.dloss, o["dZ"], o["dW"])
        tp.backward(self.block, o["dZ"], o["dX"], o["dA"], o["da"], o["dB"], o["db"])
        tp.orthogonalize(self.update["dA"], o["dA"], o["OA"])
        tp.orthogonalize(self.update["dB"], o["dB"], o["OB"])
        return o

    def status(self):
        for c in (self.block, self.head, self.update["dA"], self.update["dB"]):
            assert self.tp.check_device_status(c) == self.tp.OK


def near(got, ref, tol):
    got = got.double()
    assert bool(torch.isfinite(got).all())
    assert float((got - ref).abs().max()) <= tol * float(ref.abs().max())


def test_step_against_64_bits(tp):
    s = Step(tp, 1)
    o = s.run()
    s.status()
    Z, W, y = o["Z"].double(), s.W.double(), s.y
    S = Z @ W.t()
    lse = torch.logsumexp(S, 1)
    ok = y != -100
    at = torch.where(ok, y, 0)[:, None]
    loss = torch.where(ok, lse - S.gather(1, at)[:, 0], 0.0)
    assert torch.allclose(o["loss"].double(), loss, rtol=1e-5, atol=1e-5)
    P = torch.exp(S - lse[:, None])
    P.scatter_add_(1, at, -ok.double()[:, None])
    P *= torch.where(ok, s.dloss.double(), 0.0)[:, None]
    near(o["dZ"], P @ W, 1e-2)
    near(o["dW"], P.t() @ Z, 1e-2)
    # the block's gradients of the head's dZ
    d = {k: v.double() for k, v in s.d.items()}
    Hpre = s.block.H.double().requires_grad_()
    Y = torch.nn.functional.gelu(Hpre, approximate="tanh")
    dZ = o["dZ"].double()
    dY = torch.autograd.grad(Y, Hpre, dZ @ d["B"].t())[0]
    near(o["dA"], d["X"].t() @ dY, 2e-2)
    near(o["dB"], Y.detach().t() @ dZ, 2e-2)
    near(o["dX"], dY @ d["A"].t(), 2e-2)
    # the updates of the gradients as they are
    for G, O in (("dA", "OA"), ("dB", "OB")):
        X = o[G].double() if o[G].shape[0] <= o[G].shape[1] else o[G].double().t()
        X = X / (X.norm() + 1e-7)
        for _ in range(5):
            A = X @ X.t()
            X = 3.4445 * X + (-4.7750 * A + 2.0315 * A @ A) @ X
        X = X if o[G].shape[0] <= o[G].shape[1] else X.t()
        assert float((o[O].double() - X).norm()) <= 5e-3 * float(X.norm())


def test_step_captured_and_replayed(tp):
    s, fresh = Step(tp, 2), Step(tp, 3)
    want = {k: v.clone() for k, v in fresh.run().items()}
    s.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for k in s.d:
        s.d[k].copy_(fresh.d[k])
    s.W.copy_(fresh.W)
    s.y.copy_(fresh.y)
    for _ in range(2):
        for v in s.out.values():
            v.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(s.out[k], want[k]), k
    s.status()


def test_two_steps_at_once(tp):
    steps = [Step(tp, 4), Step(tp, 5)]
    want = [{k: v.clone() for k, v in s.run().items()} for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            for k in w:
                assert torch.equal(s.out[k], w[k]), k
    for s in steps:
        s.status()
