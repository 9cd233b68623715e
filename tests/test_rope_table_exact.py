"""The table's turns a position against the frequencies over 2 pi in exact fractions (no GPU).  Above a
radian a position an entry is rounded once, to 2^-56: 2^-57 off.  Up to one, where x is at most 0.16
turns, it is a quotient of doubles: 2 pi is off by less than 2^-54 of itself, the quotient by 2^-53 x,
the entry by 2^-57.  At the ends of int32 the angle is off by 2^-21 rad at most."""

from fractions import Fraction

import pytest

import tiled_attention_fa_gb300 as fa

# The digits of pi: 2^-262 off at most.
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def turns(f):
    """f / (2 pi), modulo 1."""
    return Fraction(f) / (2 * PI) % 1


def circle(x):
    """Distance to the nearest whole number."""
    x = x % 1
    return min(x, 1 - x)


@pytest.mark.parametrize("freqs", [
    [500000.0 ** (-2.0 * i / 128) for i in range(64)],
    [10000.0 ** (-2.0 * i / 64) for i in range(32)],
    [(-1.0) ** i * 9.0 * 0.7 ** i for i in range(32)],
    [6.2, 6.3, 12.9, 100.1, -1000.7, 54321.9, 1e9 + 0.3, -1e15 / 3],
    [1e300, -5e-324, 0.0, 2.0 ** 56, 1e-20, 3.0, -3.0, 1e18],
], ids=["base 500000", "base 10000", "mixed", "turns", "ends"])
def test_entries(freqs):
    n = len(freqs)
    words = [int(w) & (2 ** 64 - 1) for w in fa.rope_table(128, rotary=2 * n, freqs=freqs, axes=list(range(n)), device="cpu")]
    assert [w & 255 for w in words] == list(range(n))
    for w, f in zip(words, freqs):
        if abs(f) < 2.0 ** 100:  # (PI's digits)
            bound = Fraction(1, 2 ** 57) + (Fraction(abs(f)) / 6 * Fraction(3, 2 ** 54) if abs(f) <= 1 else Fraction(1, 2 ** 100))
            assert circle(Fraction(w >> 8, 2 ** 56) - turns(f)) <= bound, f


def test_base():
    """Frequencies of a base are the double base^(-2i / rotary)."""
    a = fa.rope_table(128, 500000.0, device="cpu")
    assert a.tolist() == fa.rope_table(128, freqs=[500000.0 ** (-2.0 * i / 128) for i in range(64)], device="cpu").tolist()
