"""The grouped router's exponential: the steps in the source, evaluated with exact fused multiply-adds, against 45 digits.
Its error decides how near a score has to lie to a border between two FP32 numbers for the choice to differ."""
import math
import os
import random
import re
from decimal import Decimal, getcontext
from fractions import Fraction

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fine_grained_blockwise_amd", "csrc",
                      "router_grouped.hip")


def fma(a, b, c):
    return float(Fraction(a) * Fraction(b) + Fraction(c))  # (one rounding, to nearest even)


def steps():
    """(log2 e in parts, the polynomial's coefficients, the highest power first) of the source."""
    with open(SOURCE) as f:
        text = f.read()
    body = text[text.index("double exp64("):text.index("return ldexp")]
    parts = [float(v) for v in re.findall(r"LOG2E\w* = ([\d.e+-]+)", body)]
    # as the source has it: n from the first part, r from the first and then the others
    assert "n = __builtin_rint(x * LOG2E)" in body
    assert ("r = fma(x, LOG2E_REST, fma(x, LOG2E, -n))" in body) == (len(parts) == 2) and len(parts) in (1, 2)
    coefficients = [float(v) for v in re.findall(r"(?:p = |fma\(p, r, )([\d.e+-]+)", body)]
    assert len(coefficients) == 13 and coefficients[-1] == 1.0
    return parts, coefficients


def exp64(x, parts, coefficients):
    n = float(round(x * parts[0]))
    r = fma(x, parts[0], -n)
    for part in parts[1:]:
        r = fma(x, part, r)
    p = coefficients[0]
    for c in coefficients[1:]:
        p = fma(p, r, c)
    return math.ldexp(p, int(n))


@pytest.mark.parametrize("most", [1.0, 20.0, 100.0, 200.0])
def test_exponential_is_within_two_to_the_minus_50(most):
    getcontext().prec = 45
    rng = random.Random(int(most))
    parts, coefficients = steps()
    worst = 0.0
    for x in [most, -most, 0.0] + [rng.uniform(-most, most) for _ in range(3000)]:
        e = Decimal(x).exp()
        worst = max(worst, abs(float((Decimal(exp64(x, parts, coefficients)) - e) / e)))
    assert worst <= 2.0 ** -50
