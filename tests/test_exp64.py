"""The 64-bit exponential of the verification kernels, modelled on the CPU with the
constants and the polynomial of its source: every step rounded as the device
rounds it (fma once)."""

import os
import random
import re
from decimal import Decimal, getcontext
from fractions import Fraction

from quantized_weight_skinny_amd import build as qbuild

getcontext().prec = 60
SOURCE = open(os.path.join(qbuild.CSRC, "qpn_verify.hip")).read()
BODY = SOURCE[SOURCE.index("double exp64(double x)"):SOURCE.index("return ldexp(p")]


def _constants():
    top, bottom, rest = re.search(r"kLn2 = ([\d.]+) / ([\d.]+), kLn2Rest = ([-\d.e]+);", BODY).groups()
    inverse = float(re.search(r"rint\(x \* ([\d.]+)\)", BODY).group(1))
    terms = [1.0 / float(d) for d in re.findall(r"1\.0 / (\d+\.0)", BODY)] + [0.5, 1.0, 1.0]
    return float(top) / float(bottom), float(rest), inverse, terms


def _fma(a, b, c):
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def _exp64(x):
    ln2, rest, inverse, terms = _constants()
    n = round(x * inverse)               # ties to even
    r = _fma(n, -rest, _fma(n, -ln2, x))
    p = terms[0]
    for t in terms[1:]:
        p = _fma(p, r, t)
    return Fraction(p) * Fraction(2) ** n


def test_the_two_parts_of_ln_2():
    ln2, rest, _, terms = _constants()
    assert abs(Decimal(ln2) + Decimal(rest) - Decimal(2).ln()) < Decimal(2) ** -94
    assert Fraction(ln2).denominator <= 2 ** 40                # times n <= 1155: exact in 53 bits
    assert int(800 / 0.69) * Fraction(ln2) * 2 ** 40 < 2 ** 53
    assert len(terms) == 14


def test_the_exponential_within_two_steps():
    """Half a step of the last addition, the reduction's (2^-54 of |r| <= 0.35) and the
    sum's before it (a third of a half step): below 2^-52 of the value, the result in [0.7, 1.42)."""
    rng = random.Random(1)
    for x in [0.0, -1e-300, -0.3465, -0.3466, -1.0, -745.0, -800.0] + [-rng.uniform(0, 800) for _ in range(300)] + [
            -rng.uniform(0, 2) for _ in range(300)]:
        want = Fraction(Decimal(x).exp())
        assert abs(_exp64(x) / want - 1) < Fraction(2) ** -52, x
