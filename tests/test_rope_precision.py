"""How exact the frequencies of a rotation are (CPU only): against the formulas in 60 decimal digits.

The bound, in units u = 2^-53 of f / 2 pi: the exponent -2i / R rounds once (below ln base of f), pow is below one last
place (2), 2 pi and the division by it round once each (2), a division by the scale once (1). NTK: the exponent R / (R - 2)
rounds once (1.15 |ln s| of the base), pow 2, a product 1, all to a power below 1. Together ln base + 8 + 1.2 |ln s|, base
being the scaled one. The cut to 64 bits: 2^-64 turns; a negative frequency wraps in double precision, 2^-54."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def so():
    from invariant_deterministic_bi_gb300 import _build
    _build.build()
    import invariant_deterministic_bi_gb300 as m
    return m.load()


@pytest.fixture(autouse=True)
def digits():
    old, getcontext().prec = getcontext().prec, 60
    yield
    getcontext().prec = old


def turns_of(so, R, kind, base, s, given=None):
    t, m = np.zeros(R // 2, np.uint64), ctypes.c_float()
    g = None if given is None else (ctypes.c_double * len(given))(*given)
    assert so.bi_rope_freqs(R, kind, base, s, 0, 1, 4, g, t.ctypes.data, ctypes.byref(m)) == 0
    return [Decimal(int(x)) / 2 ** 64 for x in t]


def distance(got, f):
    """Of a fraction of a turn from f / 2 pi, modulo one turn."""
    d = (f / (2 * PI) - got) % 1
    return min(abs(d), 1 - abs(d))


@pytest.mark.parametrize("R", [16, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 1000000.0, 500000.0, 1.5])
@pytest.mark.parametrize("kind,s", [(0, 1.0), (1, 8.0), (1, 0.3), (2, 4.0), (2, 32.0)])
def test_frequencies_to_double_precision(so, R, base, kind, s):
    b, scale = Decimal(base), Decimal(s)
    if kind == 2:
        b *= ((Decimal(R) / (R - 2)) * scale.ln()).exp()
    ln_b = b.ln()
    units = float(ln_b) + 8 + (1.2 * abs(math.log(s)) if kind == 2 else 0)
    for i, got in enumerate(turns_of(so, R, kind, base, s)):
        f = (-(Decimal(2 * i) / R) * ln_b).exp() / (scale if kind == 1 else 1)
        assert distance(got, f) <= Decimal(units * 2.0 ** -53) * f / (2 * PI) + Decimal(2.0 ** -64), i


def test_given_frequencies_to_double_precision(so):
    given = [1.0, -1.0, 0.75, -3e-5, 2.0 ** 20, 2.0 ** 39, -(2.0 ** 39), 1e-12]
    for f, got in zip(given, turns_of(so, 16, 5, 0, 0, given)):
        bound = 2 * 2.0 ** -53 * abs(f) / (2 * math.pi) + 2.0 ** -64 + (2.0 ** -54 if f < 0 else 0)
        assert distance(got, Decimal(f)) <= Decimal(bound), f
    assert distance(turns_of(so, 16, 5, 0, 0, given)[0], Decimal(1)) <= Decimal(2.0 ** -56)
