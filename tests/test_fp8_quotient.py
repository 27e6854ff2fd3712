"""The element quotient of the FP8 quantisers' fast path at the small end of its range, in exact
arithmetic with binary32's subnormal numbers.

Per block the device takes y = RN(1 / s) once and, for each element a, q0 = RN(a y),
r0 = RN(a - q0 s), q1 = RN(q0 + r0 y), r1 = RN(a - q1 s), q = RN(q1 + r1 y), each RN one fma.  q is
the correctly rounded a / s if r1 is exact, so r1, a multiple of ulp(q1) ulp(s), must not fall
between multiples of 2^-149, the smallest subnormal number.  E4M3's lowest rounding border is
2^-10, below which ulp(q1) = 2^-34; with s >= 2^-92, ulp(s) >= 2^-115 and r1 is exact down to it.
This exercises the method only: the library is not involved.
"""
from fractions import Fraction

import numpy as np

from tests.fp8_ref import _POS

LOWEST = -92          # the fast path's smallest scale is 2^LOWEST
TINY = Fraction(2) ** -149


def rn(x: Fraction) -> Fraction:
    """The nearest binary32 value, ties to even, subnormal numbers included."""
    if x < 0:
        return -rn(-x)
    if x == 0:
        return x
    e = x.numerator.bit_length() - x.denominator.bit_length()
    e -= Fraction(2) ** e > x
    ulp = max(Fraction(2) ** (e - 23), TINY)
    return round(x / ulp) * ulp          # (round() of a Fraction ties to even)


def quotient(a: Fraction, s: Fraction) -> Fraction:
    y = rn(1 / s)
    q0 = rn(a * y)
    q1 = rn(q0 + rn(a - q0 * s) * y)
    return rn(q1 + rn(a - q1 * s) * y)


BORDERS = [Fraction(float(lo)) / 2 + Fraction(float(hi)) / 2 for lo, hi in zip(_POS[:-1], _POS[1:])]


def _near(rng, lo, hi, count):
    """Scales in [2^lo, 2^hi) and elements on and next to E4M3's rounding borders of them."""
    for _ in range(count):
        s = Fraction(int(rng.integers(1 << 23, 1 << 24))) * Fraction(2) ** (int(rng.integers(lo, hi)) - 23)
        border = BORDERS[int(rng.integers(8 if rng.random() < 0.7 else len(BORDERS)))]
        a = rn(border * s)
        e = a.numerator.bit_length() - a.denominator.bit_length()
        e -= Fraction(2) ** e > a
        a += int(rng.integers(-3, 4)) * max(Fraction(2) ** (e - 23), TINY)
        if a > 0:
            yield a, s


def test_rounding_matches_numpy():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal(2000) * 2.0 ** rng.integers(-155, 20, 2000)).astype(np.float64)
    assert all(float(rn(Fraction(float(x)))) == float(np.float32(x)) for x in v)


def test_quotient_is_correctly_rounded_from_the_lowest_scale_on():
    rng = np.random.default_rng(1)
    for a, s in _near(rng, LOWEST, LOWEST + 6, 6000):
        assert quotient(a, s) == rn(a / s), (float(a), float(s))
    for a, s in _near(rng, LOWEST + 6, 100, 3000):
        assert quotient(a, s) == rn(a / s), (float(a), float(s))


def test_quotient_is_not_correctly_rounded_below():
    """Why the limit is there: an element on a border that would get the code above it."""
    f = lambda h: Fraction(float.fromhex(h))
    s, a, amax = f("0x1.800004p-98"), f("0x1.380004p-104"), f("0x1.500004p-89")
    assert rn(amax / 448) == s and s < Fraction(2) ** LOWEST
    assert rn(a / s) == f("0x1.ap-7") and f("0x1.ap-7") in BORDERS      # a tie: the even code
    assert quotient(a, s) == f("0x1.a00002p-7")                         # the code above
