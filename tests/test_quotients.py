"""The row quantiser's quotient by a corrected reciprocal is the correctly rounded one: all of them, in exact
arithmetic.  A cache value and a tile's largest one are bfloat16, 8 significant bits, so there are 128 x 128 pairs of
significands, and the exponents only shift the result while nothing under- or overflows."""
from fractions import Fraction


def round24(f):
    """f > 0 or f < 0 to 24 significant bits, ties to even."""
    if f == 0:
        return f
    sign, f = (-1, -f) if f < 0 else (1, f)
    e = f.numerator.bit_length() - f.denominator.bit_length()
    e += (Fraction(2) ** (e + 1) <= f) - (Fraction(2) ** e > f)
    n = f / Fraction(2) ** (e - 23)
    k, rest = n.numerator // n.denominator, n - n.numerator // n.denominator
    return sign * (k + (rest > Fraction(1, 2) or (rest == Fraction(1, 2) and k % 2))) * Fraction(2) ** (e - 23)


def test_every_pair_of_significands():
    for a in range(128, 256):
        scale = round24(Fraction(a, 448))
        r = round24(1 / scale)
        for x in range(128, 256):
            q = round24(x * r)
            left = round24(x - q * scale)             # one fused multiply-add each
            assert round24(q + left * r) == round24(x / scale), (a, x)
