"""The fixed-point angles over every frequency that a kvq_rotary may hold, against the bound that the header states."""
import os
import re
from fractions import Fraction

import numpy as np
import pytest

INV_TWO_PI = Fraction(0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E410, 1 << 192)
C, M64 = 0xA2F9836E4E44152A, (1 << 64) - 1
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvq.h")


def off(x, p):
    """How far the kernels' integer steps (a restatement) are from p x / (2 pi) turns, in turns."""
    bits = int(np.float32(abs(x)).view(np.uint32))
    ex, m = bits >> 23 & 255, (bits & 0x7FFFFF) | (0x800000 if bits >> 23 & 255 else 0)
    sh = 2 - ((ex or 1) - 150)
    u = ((m * C >> sh) if sh >= 0 else m * C << -sh) & M64
    u = -u & M64 if x < 0 else u
    ul, uh, up = u & 0xFFFFFFFF, u >> 32, p & 0xFFFFFFFF
    top = ((ul * up >> 32) + uh * up - (ul if p < 0 else 0)) & 0xFFFFFFFF
    turn = Fraction(top, 1 << 32) - Fraction(float(x)) * p * INV_TWO_PI
    return abs(turn - round(turn))


def stated():
    """(bound below 2 radians per position, bound below 2^16), as powers of two."""
    text = re.sub(r"[\s*]+", " ", open(HEADER, encoding="utf-8").read())
    got = re.search(r"exact to 2\^-(\d+) of a turn at any 32-bit position for \|inv_freq\| below 2, and to 2\^-(\d+) below 2\^16", text)
    assert got, "the header states no such bound"
    return tuple(Fraction(1, 1 << int(x)) for x in got.groups())


@pytest.mark.parametrize("lo,hi", [(-40, 0), (0, 1), (1, 8), (8, 15.9), (15, 16)])
def test_stated_bound_holds(lo, hi):
    """Cut at 2^-32 of a turn.  Beside that p, 2^31 at most, times the error of a position's turns: 2^-64 for their own cut and
    0.0151 of that (what the rounded constant is off by) for each unit of the 24-bit fraction that it is multiplied by, over
    2^25 (f below 2: less than one) or 2^10 (below 2^16: 247): 1.5 * 2^-32 and 2^-25 + 2^-32 together."""
    small, large = stated()
    r = np.random.Generator(np.random.PCG64(7))
    f = np.float32(2.0) ** r.uniform(lo, hi, 400).astype(np.float32)
    f = np.minimum(f, np.nextafter(np.float32(2.0 ** hi), np.float32(0)))
    for x in f:
        for p in (1, -1, 131071, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31, int(r.integers(-2 ** 31, 2 ** 31))):
            for s in (1.0, -1.0):
                assert off(s * float(x), p) <= (small if x < 2 else large), (x, p)
