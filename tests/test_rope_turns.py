"""Turns per position against 60 digits, without a GPU: to half a unit of 2^-64, so that far positions keep their angles."""
import ctypes
import math
from decimal import Decimal, getcontext

import pytest


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import build
    build.build()
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


@pytest.fixture(autouse=True)
def digits():
    before, getcontext().prec = getcontext().prec, 60
    yield
    getcontext().prec = before


def two_pi():
    """Machin: pi = 16 arctan(1/5) - 4 arctan(1/239)."""
    def arctan(n):
        x, total, k = Decimal(1) / n, Decimal(0), 0
        while abs(x) > Decimal(10) ** -62:
            total += (-1) ** k * x / (2 * k + 1)
            x, k = x / (n * n), k + 1
        return total
    return 2 * (16 * arctan(5) - 4 * arctan(239))


def turns_of(base, rot, scaling=None):
    """theta_i / (2 pi), exact."""
    out, whole = [], two_pi()
    for i in range(rot // 2):
        f = (Decimal(base).ln() * (-2 * i) / rot).exp()
        if scaling and scaling[0] == "linear":
            f /= Decimal(scaling[1])
        elif scaling:
            _, factor, context, low, high = (Decimal(x) if not isinstance(x, str) else x for x in scaling)
            k = min(Decimal(1), max(Decimal(0), (context * f / whole - low) / (high - low)))
            f *= k + (1 - k) / factor
        out.append(f / whole)
    return out


@pytest.mark.parametrize("rot", [2, 48, 64, 96, 128, 256])
@pytest.mark.parametrize("base", [1.0, 1.0 + 2.0 ** -30, 1.5, 10000.0, 500000.0, 1e300, 1.7e308])
@pytest.mark.parametrize("scaling", [None, ("linear", 3.7), ("parts", 8.0, 2048, 1.0, 32.0), ("parts", 40.0, 4096, 0.3, 17.1),
                                     ("parts", 4.0, 1 << 40, -1.7e308, 1.7e308), ("parts", 4.0, 1, 5.0, 5.0 + 2.0 ** -50)])
def test_turns(tp, base, rot, scaling):
    table = tp.RopeTable(rot, base, scaling=scaling, device="cpu")
    for got, want in zip(table.turns.tolist(), turns_of(base, rot, scaling)):
        # two doubles hold 2^-80 of a turn; the rounding is half a unit
        assert abs(Decimal(got % 2 ** 64) - want * 2 ** 64) <= Decimal(0.5) + Decimal(2) ** -10


def test_close_to_a_whole_turn(tp):
    """factor stretches pair 0 to just below 2 pi; no more than a turn is accepted."""
    inverse = 1 / two_pi()
    nearest = float(inverse)
    above = nearest if Decimal(nearest) > inverse else math.nextafter(nearest, 1.0)
    r = tp.Rope(10000.0, above, 0.0, 1.0, 1, 2, tp.ROPE_SCALE_LINEAR)
    out = (ctypes.c_uint64 * 1)()
    assert tp.lib.tpmlp_rope_turns(ctypes.byref(r), out) == tp.OK
    assert abs(Decimal(out[0]) - 2 ** 64 / (two_pi() * Decimal(above))) <= Decimal(0.5) + Decimal(2) ** -10
    r.factor = math.nextafter(above, 0.0)
    assert tp.lib.tpmlp_rope_turns(ctypes.byref(r), out) == tp.ERR_INVALID_ARG
