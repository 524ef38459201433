"""Frequencies as whole numbers of 2^-64 turns against rational arithmetic: rounded to the nearest, whole turns left out."""
from fractions import Fraction

import pytest
import torch

import hybrid_linear_attention_decode_gb300 as kda

# pi to 50 digits, so that 2^64 theta / 2 pi is known to far below one
PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


@pytest.fixture(scope="module", autouse=True)
def built():
    from hybrid_linear_attention_decode_gb300 import build as kbuild
    kbuild.build()


def turns(rope):
    return [int(t) % (1 << 64) for t in rope.turns.tolist()]


def exact(theta):
    """2^64 theta / 2 pi of a double, whole turns left out."""
    x = Fraction(theta) / (2 * PI)
    return (x - x.numerator // x.denominator) * (1 << 64)


def check(got, theta, ulps):
    """A unit of 2^-64 is rounded to the nearest: off by half.  theta / 2 pi in doubles: 2 pi and the quotient are off by
    at most half a step each, 2^-53 of the value, and `ulps` more such steps are in theta itself."""
    for g, t in zip(got, theta, strict=True):
        x = Fraction(t) / (2 * PI)
        off = abs(g - exact(t))
        off = min(off, (1 << 64) - off)  # just below a whole turn and just above are neighbours
        assert off <= Fraction(1, 2) + (2 + ulps) * x * (1 << 64) / (1 << 53), (t, float(off))


def test_given_frequencies():
    g = torch.Generator().manual_seed(0)
    e = torch.rand(2000, generator=g, dtype=torch.float64) * 84 - 64  # 2^-64 to 2^20
    theta = [0.0, 2.0 ** -70, 6.2831853071795862, 3.1415926535897931, 2.0 ** 20 - 1] + (2.0 ** e).tolist()
    check(turns(kda.Rope.of(theta, device="cpu")), theta, 0)


@pytest.mark.parametrize("base", [1.0, 100.0, 10000.0, 500000.0, 1e8, 1e30])
def test_of_a_base(base):
    # pow is off by one step at most, and so is its argument's part (|log theta| below 70 steps of it)
    theta = [base ** (-2.0 * i / 128) for i in range(64)]
    check(turns(kda.Rope.make(128, base, device="cpu")), theta, 2)
    check(turns(kda.Rope.make(128, base, scaling="linear", factor=32.0, device="cpu")), [t / 32 for t in theta], 2)


def test_far_positions_of_low_frequencies():
    """At position 2^31 an angle is off by the frequency's half unit 2^31 times: 2^-34 of a turn, not 2^-33."""
    theta = [2.0 ** -41 * (1 + i / 1000) for i in range(1000)]
    for g, t in zip(turns(kda.Rope.of(theta, device="cpu")), theta):
        assert abs((1 << 31) * (g - exact(t))) <= (1 << 30) * (1 + 2.0 ** -20)
