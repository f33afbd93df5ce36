"""Rows whose codes lie as near to a tie as float32 values allow, by construction.

With v / a = 2^e V / A (V, A whole, of 24 bits) and e <= 0, the distance of 127
v / a from c + 1/2 is |254 V - (2c + 1) A 2^-e| / (2 A 2^-e): a whole number,
even where e < 0, over 2 A 2^-e. ``rows`` solves for the smallest ones, on both
sides of the tie, beside exact ties of the same rows."""
import math

import numpy as np

# code below the tie, exponent of v / a: ties from 1/2 to the largest
PLACES = [(0, -8), (0, -7), (1, -6), (2, -5), (5, -4), (10, -3), (21, -2), (42, -1), (62, -1), (100, 0), (126, 0)]


def _nearest(c, e, off):
    """The largest 24-bit A with a 24-bit V for which 254 V = (2c + 1) A 2^-e + off."""
    s = (2 * c + 1) << -e
    for first in range(254):
        if (s * first + off) % 254 == 0:
            a = first + 254 * ((2 ** 24 - 1 - first) // 254)
            while a >= 2 ** 23:
                v = (s * a + off) // 254
                if 2 ** 23 <= v < 2 ** 24:
                    return a, v
                a -= 254
    return None


def rows(exponent=0):
    """float32 rows [a, v, -v, a/2, -a/2, 0, ...], all times 2^exponent: v next to a tie, a/2 (63.5 steps) on one."""
    out = []
    for c, e in PLACES:
        for off in (1, -1, 2, -2):
            if off % 2 and e < 0:
                continue  # the difference is even
            got = _nearest(c, e, off)
            if got is None:
                continue
            a, v = got
            out.append([a, v * 2.0 ** e, -v * 2.0 ** e, a / 2, -a / 2, 0, 1, -1])
    r = np.ldexp(np.array(out), exponent)
    assert np.array_equal(r, r.astype(np.float32))  # every value is a float32
    return r.astype(np.float32)


def nearest_distance(r):
    """log2 of the smallest distance from a tie that is none, over the rows (exact)."""
    from fractions import Fraction

    least = min(abs(127 * Fraction(float(row[1])) / Fraction(float(row[0])) % 1 - Fraction(1, 2)) for row in r)
    assert least > 0
    return math.log2(least)
