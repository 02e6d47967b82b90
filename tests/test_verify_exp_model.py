"""The exponential of the verification kernels (csrc/amk_op_verify.cu, exp_neg)
replayed in Python on the constants of its source, against the exact one."""
import math
import os
import re
from fractions import Fraction

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def constants():
    src = open(os.path.join(ROOT, "persistent_megakernel_decode_cta_b200", "csrc",
                            "amk_op_verify.cu")).read()
    hi, lo = re.search(r"kHi = (0x[0-9a-fp.+-]+), kLo = (0x[0-9a-fp.+-]+);", src).groups()
    scale = re.search(r"fma\(y, ([0-9.]+), 6755399441055744.0\)", src).group(1)
    return float.fromhex(hi), float.fromhex(lo), float(scale)


def fma(a, b, c):  # one rounding
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def exp_neg(y, hi, lo, scale):
    if not y > -700.0:
        return 0.0
    n = round(Fraction(y) * Fraction(scale))
    f = float(n)
    r = fma(f, -lo, fma(f, -hi, y))
    assert abs(r) <= math.log(2) / 128 * (1 + 1e-9)
    q = fma(r, 1.0 / 120, 1.0 / 24)
    q = fma(r, q, 1.0 / 6)
    q = fma(r, q, 0.5)
    q = fma(r, q, 1.0)
    t = 2.0 ** ((n & 63) / 64.0)
    return math.ldexp(fma(t * r, q, t), n >> 6)


def test_within_two_units_in_the_last_place():
    """The series' cut is below 2^-57 of the value, the table and the two last
    roundings half a unit each, the first product's rounding 2^-7 of one."""
    k = constants()
    ys = [-i * 0.001 for i in range(1, 2000)] + [-i * 0.37 for i in range(1, 1890)] + \
         [-1e-300, -1e-17, -2.0**-30, -699.999, 0.0, -0.0]
    worst = 0.0
    for y in ys:
        want, got = math.exp(y), exp_neg(y, *k)
        worst = max(worst, abs(got - want) / math.ulp(want))
    assert worst <= 2.0, worst
    assert exp_neg(0.0, *k) == 1.0
