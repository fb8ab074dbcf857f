"""The fp32 form of the quantisers' division (dg_quant.h, divide) gives the E4M3
codes of the IEEE quotient, for every x and every scale.

With z = x / s, y = RN(1/s), q0 = RN(x y), e = RN(q0 s - x) (one fma) and
q = RN(q0 - e y) (one fma): y is 1/s (1 + d1) and e is s (q0 - z) (1 + d2) with
|d1|, |d2| <= 2^-24, and |q0 - z| <= 1.5 ulp(z) up to 2^-24 of it.  So what the
last step rounds is z - (q0 - z)(d1 + d2 + d1 d2), within D = 1.5 * 2^-23 ulp(z)
(1 + 2^-20) of z.  Unless a midpoint of fp32 lies within D of z, q = RN(z); if
one does, q and RN(z) are the two fp32 values next to it.  A code changes at
its boundaries m, which are fp32 values of at most five bits, so the two values
differ in their codes only if one of them is m itself: z is within D of
m +- ulp / 2.

Let m = M 2^k with 16 <= M < 32 and s = S 2^a with 2^23 <= S < 2^24.  In units
of 2^(k+a), s ulp / 2 is S 2^-20 and x an integer (its unit is 16 or 32, since
M S is at least 2^27), so x - M S = +-c with S 2^-20 within 1.5 * 2^-18 of the
integer c: S = c 2^20 + j with |j| <= 6.  Below a power of two (M = 16) ulp is
half as large and S = c 2^21 + j.  That is a finite list, and it is checked
here one by one in exact arithmetic; powers of two in x and s change nothing
while nothing underflows: |x| >= 2^-11 s and s >= 1e-4 / 448 keep every
intermediate above 2^-60, and s <= 2^128 / 448 keeps y normal."""
import random
from fractions import Fraction

import pytest


def exponent(v):
    """floor(log2 v) of a positive fraction."""
    e = v.numerator.bit_length() - v.denominator.bit_length()
    return e if v >= Fraction(2) ** e else e - 1


def rn(v, bits=24):
    """v rounded to `bits` significant bits, ties to even."""
    if v == 0:
        return v
    unit = Fraction(2) ** (exponent(abs(v)) - bits + 1)
    return round(v / unit) * unit                      # Python rounds halves to even


def divide(x, s):
    y = rn(1 / s)
    q0 = rn(x * y)
    e = rn(q0 * s - x)
    return rn(q0 - e * y)


def candidates():
    for M in range(16, 32):
        for sign, shift in ((1, 20), (-1, 20)) if M > 16 else ((1, 20), (-1, 21)):
            for c in range(1, 17):
                for j in range(-8, 9):
                    S = c * 2 ** shift + j
                    if not 2 ** 23 <= S < 2 ** 24:
                        continue
                    x = M * S + sign * c
                    if x % 2 ** (x.bit_length() - 24) == 0:
                        yield Fraction(M), Fraction(S), Fraction(x)


def test_codes_next_to_every_boundary():
    seen = close = 0
    for m, s, x in candidates():
        want, got = rn(x / s), divide(x, s)
        # the same side of the boundary, or both on it: the same code, whichever way the tie goes
        assert (got > m) - (got < m) == (want > m) - (want < m), (m, s, x)
        seen += 1
        ulp = Fraction(2) ** (exponent(x / s) - 23)
        close += abs(abs(x / s - m) - ulp / 2) <= Fraction(3, 2 ** 24) * ulp
    assert seen > 100 and close > 20, (seen, close)     # the list does hold such quotients


def test_the_bounds_of_the_derivation():
    """q0 within 1.5 ulp (up to 2^-24 of it), what the last step rounds within D, on random pairs; and quotients that show
    that q0 may be more than an ulp off and e inexact."""
    rng = random.Random(1)
    far = inexact = 0
    for _ in range(20000):
        s, x = Fraction(rng.randrange(2 ** 23, 2 ** 24)), Fraction(rng.randrange(2 ** 23, 2 ** 24))
        if rng.random() < 0.5:
            x = Fraction(int(s * Fraction(rng.randrange(900, 1000), 1000)))
        z, y = x / s, rn(1 / s)
        ulp = Fraction(2) ** (exponent(z) - 23)
        q0 = rn(x * y)
        e = rn(q0 * s - x)
        assert abs(q0 - z) <= Fraction(3, 2) * ulp * (1 + Fraction(1, 2 ** 23))
        assert abs(q0 - e * y - z) <= Fraction(3, 2 ** 24) * ulp * (1 + Fraction(1, 2 ** 20))
        assert divide(x, s) == rn(z)
        far += abs(q0 - z) > ulp
        inexact += e != q0 * s - x
    assert far and inexact


@pytest.mark.parametrize("m", [Fraction(17), Fraction(16), Fraction(31)])
def test_a_planted_error_is_seen(m):
    """The comparison tells a quotient that landed on the boundary from one beside it."""
    beside = m + Fraction(2) ** (exponent(m) - 23)
    assert (beside > m) - (beside < m) != (m > m) - (m < m)
