"""The kernels' reduction of rotary angles, restated in whole numbers and fp32 (CPU): at every
int32 position the fraction of a turn is that of p f / (2 pi) in many more bits, to
within what the documented error of cos and sin, 2^-20, leaves beside the two
functions' own (some 2^-22)."""
import random
import struct
from fractions import Fraction

import numpy as np
import pytest

PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
HI, LO = 0xA2F9836E, 0x4E441529
M64 = (1 << 64) - 1


def test_two_over_pi():
    assert (HI << 32 | LO) == int((1 << 64) * 2 / PI)


def rate_of(f):
    bits = struct.unpack("<I", struct.pack("<f", f))[0]
    m = (bits & 0x7FFFFF) << 8 | 0x80000000
    x = (m * HI + (m * LO >> 32)) & M64
    down = 128 - (bits >> 23 & 255)
    r = 0 if abs(down) >= 64 else x >> down if down >= 0 else x << -down & M64
    return -r & M64 if bits >> 31 else r


def half_turns(pos, rate):
    t = (pos * rate & M64) >> 32
    return float(np.float32(t - (1 << 32) if t >> 31 else t) * np.float32(2.0 ** -31))


def off(pos, f):
    """Error of the angle, in radians."""
    exact = 2 * (pos * Fraction(f) / (2 * PI))             # half turns
    d = (Fraction(half_turns(pos, rate_of(f))) - exact) % 2
    return float(min(d, 2 - d) * PI)


@pytest.mark.parametrize("top", [1, 8, 16, 24, 26, 27, 28, 29, 30, 31])
@pytest.mark.parametrize("far", [1.0, 1e-3, 1e-7])
def test_positions(top, far):
    rnd = random.Random(top)
    at = [rnd.randrange(1 << (top - 1), 1 << top) for _ in range(300)] + [(1 << top) - 1, 1 << (top - 1)]
    worst = max(off(s * p, float(np.float32(g * far))) for p in at
                for g in (1.0, rnd.uniform(0.25, 1.0), -rnd.uniform(0.25, 1.0)) for s in (1, -1))
    # an fp32 number of half turns below 1 is off by 2^-25, what is cut off by 2^-31 of them
    assert worst < (2.0 ** -25 + 2.0 ** -31) * 3.1416 + 2.0 ** -31


def test_ends():
    for f in (0.0, 1.0, -1.0, 2.0 ** -126, 1e-45, 1.9999999, 2.0, 1000.0):
        f = float(np.float32(f))
        for p in (0, 1, -1, 2 ** 31 - 1, -2 ** 31):
            assert off(p, f) < 2.0 ** -20 * max(1.0, abs(f) / 64), (p, f)
