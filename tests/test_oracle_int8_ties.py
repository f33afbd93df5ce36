"""The 8-bit oracle next to ties, and on rows whose scale is subnormal, against
exact rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

import int8_ties
from oracle import int8 as OI


@pytest.mark.parametrize("exponent", [0, -24, 60, -120])
def test_codes_next_to_ties(exponent):
    v = int8_ties.rows(exponent)
    # as near as float32 values come: over 2^-32, and within twice of it
    assert len(v) >= 20 and -32 < int8_ties.nearest_distance(v) < -31
    codes, _ = OI.quantize(v)
    a = [Fraction(float(row[0])) for row in v]
    want = [[round(127 * Fraction(float(t)) / a[i]) for t in row] for i, row in enumerate(v)]
    assert codes.tolist() == want
    # what one product with the rounded reciprocal gives is wrong here
    short = np.rint(v[:, 1] * (np.float32(127) / v[:, 0]))
    assert (short != codes[:, 1]).any()


def _fl32(q):
    """A positive Fraction rounded to float32's grid, ties to even, subnormals included."""
    e = -149
    while q / Fraction(2) ** e >= 2 ** 24:
        e += 1
    return float(round(q / Fraction(2) ** e) * Fraction(2) ** e)


@pytest.mark.parametrize("exponent", [0, -30, -80, -120, -125, -130, -140, -148])
def test_scales_equal_rational_rounding(exponent):
    rng = np.random.default_rng(-exponent)
    v = (rng.standard_normal((300, 3)) * 2.0 ** exponent).astype(np.float32)
    v[0] = 2.0 ** -149
    v[1] = 127 * 2.0 ** -149
    v[2] = 190 * 2.0 ** -149  # 1.496 steps of the subnormals
    v[3] = 63 * 2.0 ** -149
    v[4] = 64 * 2.0 ** -149
    _, scale = OI.quantize(v)
    for i in range(len(v)):
        a = max(abs(Fraction(float(t))) for t in v[i])
        assert float(scale[i]) == (_fl32(a / 127) if a else 0.0)
    assert scale[0] == scale[3] == 0 and scale[1] == scale[2] == scale[4] == np.float32(2.0 ** -149)
