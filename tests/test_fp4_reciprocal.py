"""The NV quantisation's division by a block scale, x r + x rest, in exact
arithmetic: its code at every midpoint of e2m1 and both fp32 neighbours,
under every e4m3 scale, for matrix scales at the ends of their range, where
`rest` is subnormal.  Independent of the approximate reciprocal's last bit."""

from fractions import Fraction as F

import numpy as np
import pytest

E4M3 = [(b & 7) * F(1, 512) if b < 8 else (8 + (b & 7)) * F(2) ** ((b >> 3) - 10) for b in range(127)]
E2M1 = [F(0), F(1, 2), F(1), F(3, 2), F(2), F(3), F(4), F(6)]
LARGEST = F(float(np.finfo(np.float32).max))


def nearest(x: F) -> F:
    """x rounded to fp32 (range above not limited), ties to even, subnormals included."""
    if x == 0:
        return x
    a = abs(x)
    e = a.numerator.bit_length() - a.denominator.bit_length()
    e -= F(2) ** e > a
    unit = F(2) ** (max(e, -126) - 23)
    n, rest = divmod(a, unit)
    n += rest * 2 > unit or (rest * 2 == unit and n & 1)
    return n * unit * (1 if x > 0 else -1)


def neighbours(x: F):
    unit = nearest(x)
    f = np.float32(float(unit))
    return [unit, F(float(np.nextafter(f, np.float32(0))))] + (
        [F(float(np.nextafter(f, np.float32(np.inf))))] if unit < LARGEST else [])


def down(x: F) -> F:
    y = nearest(x)
    return y if y <= x else F(float(np.nextafter(np.float32(float(y)), np.float32(-np.inf))))


def code(q: F) -> int:
    return min(range(8), key=lambda i: (abs(E2M1[i] - q), i & 1))


@pytest.mark.parametrize("e", [-100, 0, 100, 110, 115, 116, 117])
def test_codes_at_midpoints(e):
    g = F(2) ** e
    for s in E4M3[1:]:
        d = s * g
        if s > nearest(LARGEST / (6 * g)) * F(33, 32):  # past the scale of the largest finite magnitude, rounded up
            continue
        for a in neighbours(1 / d):
            r = down(nearest(1 - d * a) * a + a)
            rest = nearest(nearest(1 - d * r) * r)
            assert r >= 0 and rest >= 0
            for i in range(7):
                for x in neighbours((E2M1[i] + E2M1[i + 1]) / 2 * d):
                    if x <= LARGEST:
                        q = nearest(x * r + nearest(x * rest))
                        assert code(q) == code(x / d), (float(s), float(x))
