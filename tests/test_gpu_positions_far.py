"""Angles of far positions on the GPU against 60 digits: off by 2^-26 + 2^-32 + |position| 2^-65 of a turn at most, the sine and
cosine by a step of 2^-24 of their own."""
import math
from decimal import Decimal

import pytest
import torch

from test_rope_turns import digits, turns_of, two_pi  # noqa: F401 (digits: a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def angle(turn):
    """sin and cos of a number of turns in 60 digits."""
    f = turn - turn.to_integral_value()
    x = float(f * two_pi())
    return math.cos(x), math.sin(x)


@pytest.mark.parametrize("scaling", [None, ("parts", 8.0, 2048, 1.0, 32.0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(tp, layout, scaling):
    d = 64
    places = [n for e in range(24, 46, 3) for n in (2 ** e, 2 ** e + 12345, -3 * 2 ** (e - 1) - 7)]
    T = len(places)
    pos = torch.tensor(places, device="cuda")
    Q, K = torch.zeros(T, 1, d, device="cuda"), torch.zeros(T, 1, d, device="cuda")
    first = slice(0, d // 2) if layout == "half" else slice(0, d, 2)
    second = slice(d // 2, d) if layout == "half" else slice(1, d, 2)
    Q[..., first] = 1.0  # a pair (1, 0) becomes (cos, sin)
    ctx = tp.QkContext(T, 1, 1, d, torch.float32, tp.RopeTable(d, 500000.0, layout, scaling), norm=False)
    Qr, _ = tp.qk_forward(ctx, (Q, K), pos)
    c, s = Qr[:, 0, first].double().cpu(), Qr[:, 0, second].double().cpu()
    for i, turn in enumerate(turns_of(500000.0, d, scaling)):
        for j, n in enumerate(places):
            tol = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32 + abs(n) * 2.0 ** -65) + 2.0 ** -24
            want = angle(Decimal(n) * turn)
            assert abs(float(c[j, i]) - want[0]) <= tol and abs(float(s[j, i]) - want[1]) <= tol, (n, i)
