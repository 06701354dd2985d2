"""The block quantiser's quotients: one product with the scale's reciprocal,
corrected by one residual, is the IEEE quotient for every pair of a value's
and a block maximum's bf16 significand (their exponents only shift it).  In
exact rational arithmetic, each operation rounded to 24 bits."""
from fractions import Fraction

E4M3_MAX = 448


def _rn24(x: Fraction) -> Fraction:
    """x rounded to 24 significant bits, ties to even."""
    if x == 0:
        return x
    sign, x = (-1, -x) if x < 0 else (1, x)
    e = x.numerator.bit_length() - x.denominator.bit_length()
    if Fraction(2) ** e > x:
        e -= 1
    unit = Fraction(2) ** (e - 23)
    n, rest = divmod(x, unit)
    n = int(n) + (1 if rest * 2 > unit or (rest * 2 == unit and int(n) & 1) else 0)
    return sign * n * unit


def _corrected(v, s, y):
    q = _rn24(v * y)
    return _rn24(q - _rn24(q * s - v) * y)


def test_every_pair_of_significands():
    inv = _rn24(Fraction(1, E4M3_MAX))
    for top in range(128, 256):
        scale = _rn24(Fraction(top, E4M3_MAX))
        assert _corrected(Fraction(top), Fraction(E4M3_MAX), inv) == scale, top
        y = _rn24(1 / scale)
        for sig in range(128, 256):
            v = Fraction(sig)
            assert _corrected(v, scale, y) == _rn24(v / scale), (top, sig)
