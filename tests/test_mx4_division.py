"""The three-instruction division of nvfp4 quantisation, emulated with exact fractions: with a
reciprocal that is off by up to an ulp, its result and the correctly rounded quotient lie on the
same side of every boundary, except for divisors whose significand is next to a multiple of 2^22
(codes) or 2^20 (block scales), but not at one.  Those take a real division."""
import random
from fractions import Fraction as F

import pytest

CODES = [F(1, 4), F(3, 4), F(5, 4), F(7, 4), F(5, 2), F(7, 2), F(5)]
# Boundaries of e4m3: midpoints of its normal numbers (one binade), and of its subnormal ones.
SCALES = [F(m, 16) for m in range(17, 32, 2)] + [F(m, 1024) for m in range(1, 16, 2)]


def ulp(v):
    v = abs(v)
    e = v.numerator.bit_length() - v.denominator.bit_length()
    if F(2) ** e > v:
        e -= 1
    return F(2) ** (e - 23)


def fp32(v):
    """v rounded to 24 bits, ties to even."""
    if v == 0:
        return v
    n, u = v / ulp(v), ulp(v)
    low = n.numerator // n.denominator
    rest = n - low
    return (low + (rest > F(1, 2) or (rest == F(1, 2) and low % 2 == 1))) * u


def divide(x, d, r):
    q = fp32(x * r)
    return fp32(q - fp32(q * d - x) * r)


def misjudged(significand, boundaries):
    """Boundaries that some number next to them falls to another side of, for some reciprocal."""
    d = F(significand, 2 ** 23)
    near = fp32(1 / d)
    u = ulp(near)
    reciprocals = {r for r in (near - u, near - u / 2, near, near + u / 2, near + u)
                   if abs(r - 1 / d) <= u and fp32(r) == r}
    bad = []
    for m in boundaries:
        base = fp32(m * d)
        for k in range(-3, 4):
            x = fp32(base + k * ulp(base))
            want = fp32(x / d)
            for r in reciprocals:
                got = divide(x, d, r)
                if (got > m) != (want > m) or (got < m) != (want < m):
                    bad.append((m, k))
    return bad


def judges(significand, modulus):
    """As in the kernels."""
    low = significand % modulus
    return low == 0 or (low + 32) % modulus > 64


def divisors(modulus):
    near = [base + j for base in range(2 ** 23, 2 ** 24 + 1, modulus) for j in range(-44, 45, 4 if modulus < 2**22 else 1)
            if 2 ** 23 <= base + j < 2 ** 24]
    rng = random.Random(modulus)
    return near + [rng.randrange(2 ** 23, 2 ** 24) for _ in range(300)]


@pytest.mark.parametrize("modulus,boundaries", [(2 ** 22, CODES), (2 ** 20, SCALES)])
def test_no_boundary_is_misjudged(modulus, boundaries):
    for significand in divisors(modulus):
        if judges(significand, modulus):
            assert not misjudged(significand, boundaries), hex(significand)


def test_excluded_divisors_are_needed():
    """A number of 1.25 scales whose quotient comes out as the one below: code 1, not 1.5."""
    assert misjudged(0xFFFFFC, CODES) and not judges(0xFFFFFC, 2 ** 22)
    d, x, r = F(0xFFFFFC, 2 ** 23), F(0x9FFFFE, 2 ** 22), F(0x800003, 2 ** 24)
    assert abs(r - 1 / d) <= ulp(r) and fp32(x / d) > F(5, 4) and divide(x, d, r) == F(5, 4)


def test_scales_of_one_are_fast():
    """Without a tensor scale no divisor is excluded: e4m3 has four significant bits."""
    assert all(judges(m << 20, 2 ** 22) for m in range(8, 16)) and judges(6 << 21, 2 ** 20)
