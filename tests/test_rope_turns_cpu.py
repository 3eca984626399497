"""FARope.new's turns against quotients by pi in exact fractions."""
import random
from fractions import Fraction

import pytest

import attention_forward_02_gb300 as fa

# 400 decimals of pi by Euler's series, apart from the formula that the package uses: with y = x^2 / (1 + x^2)
# arctan x = y / x (1 + 2/3 y + 2 4 / (3 5) y^2 + ...), and pi = 20 arctan(1 / 7) + 8 arctan(3 / 79)


def euler(x, places):
    """arctan of a Fraction, to 10^-places."""
    y = x * x / (1 + x * x)
    term, total, k = y / x, Fraction(0), 0
    small = Fraction(1, 10 ** places)
    scale = 10 ** (places + 20)
    while term > small:
        total += term
        k += 1
        term = Fraction(int(term * y * Fraction(2 * k, 2 * k + 1) * scale), scale)
    return total


PI = 20 * euler(Fraction(1, 7), 400) + 8 * euler(Fraction(3, 79), 400)


def exact(x):
    return Fraction(x) / (2 * PI) * 2 ** 64


def off(got, x):
    """Distance in units of 2^-64 of a turn, whole turns aside."""
    d = (got - exact(x)) % 2 ** 64
    return min(d, 2 ** 64 - d)


def test_pi():
    digits = "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651"
    assert abs(PI - Fraction(digits)) < Fraction(1, 10 ** 109)


@pytest.mark.parametrize("rot,base,scaling", [(128, 10000.0, None), (128, 500000.0, "yarn"), (64, 1e6, "bands"),
                                              (32, 10000.0, "linear"), (128, 10000.0, "base"), (8, 1e12, None)])
def test_frequencies(rot, base, scaling):
    from attention_forward_02_gb300.rope import _scaled
    w, _ = _scaled(rot, base, scaling, 8.0, 8192, 32.0, 1.0)
    turns = fa.FARope.new(rot, base=base, scaling=scaling, trained=8192, device="cpu").turns.tolist()
    assert max(off(t, x) for t, x in zip(turns, w)) <= Fraction(1, 2) + Fraction(1, 10 ** 9)


def test_any_radians():
    rng = random.Random(0)
    x = [rng.choice([-1, 1]) * rng.random() * 2.0 ** rng.randint(-80, 300) for _ in range(400)]
    x += [0.0, -0.0, 1e-300, -5e-324, 2.0 ** 500, -(2.0 ** 500) * 1.1, 3.141592653589793, 6.283185307179586, -3.141592653589793,
          1.0, -1.0, 2.0 ** -64]
    turns = fa.FARope.new(2 * len(x) // 8 * 8, radians=x[:len(x) // 4 * 4], device="cpu").turns.tolist()
    for t, y in zip(turns, x):
        assert -2 ** 63 <= t < 2 ** 63 and off(t, y) <= Fraction(1, 2) + Fraction(1, 10 ** 9), y
