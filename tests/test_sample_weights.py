"""How near sampling's fixed-point weights are to the exponentials they stand
for: the kernel's arithmetic, step by step in numbers that are rounded where
the GPU rounds, against 60 decimal digits.  libscan.h states the bound."""
import math
import random
from decimal import Decimal, getcontext
from fractions import Fraction

getcontext().prec = 60
POWERS = 512
LN2 = Decimal(2).ln()


def fma(a, b, c):
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def exact_power(i):
    """2^(i / 512) to the nearest double."""
    return float((LN2 * i / POWERS).exp())


def word(x, top, temperature, shift):
    """The weight of x as sample_kernels.hip makes it."""
    by = POWERS * 1.4426950408889634074 / temperature
    d = float(x) - float(top)
    magic = 6755399441055744.0
    t = fma(d, by, magic)
    k = int(Fraction(t) - Fraction(magic))
    r = fma(d, by, magic - t)
    c = 0.6931471805599453094 / POWERS
    p = fma(r, c * c * c / 6, c * c / 2)
    p = fma(p, r, c)
    p = fma(p, r, 1.0)
    scale = math.ldexp(exact_power(k % POWERS), shift + k // POWERS)
    return int(Fraction(fma(scale, p, 4503599627370496.0)) - 4503599627370496)


def test_weights_are_within_the_stated_bound():
    rng = random.Random(1)
    single = lambda v: float(Fraction(int(v * 2 ** 20), 2 ** 20))  # noqa: E731
    worst = 0.0
    for shift in (38, 45, 51):
        for _ in range(1500):
            top, temperature = single(rng.uniform(-30, 30)), single(rng.choice((0.1, 0.7, 1.0, 3.0)) * rng.uniform(0.5, 1.5))
            x = top - single(temperature * rng.uniform(0, 37) ** rng.choice((1, 0.3)))
            want = ((Decimal(x) - Decimal(top)) / Decimal(temperature)).exp() * 2 ** shift
            off = abs(Decimal(word(x, top, temperature, shift)) - want)
            assert off <= Decimal(0.5) + want * Decimal(2) ** -45, (x, top, temperature, shift)
            worst = max(worst, float(off))
    # and not to the nearest word
    assert worst > 1.0


def test_the_largest_is_one():
    for shift in (38, 51):
        assert word(3.25, 3.25, 0.7, shift) == 1 << shift
