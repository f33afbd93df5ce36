"""The 8-bit and clipping oracles against exact rational arithmetic."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import clip as OC
from oracle import int8 as OI


def _half_even(q: Fraction) -> int:
    return round(q)  # Python rounds a Fraction half to even


@pytest.mark.parametrize("kind", ["normal", "bf16_grid", "tiny", "halves"])
def test_codes_equal_rational_rounding(kind):
    rng = np.random.default_rng(7)
    v = rng.standard_normal((6, 50)).astype(np.float32)
    if kind == "bf16_grid":  # many exact ties: half the largest magnitude is 63.5 steps
        v = (np.rint(v * 16) / 16).astype(np.float32)
        v[:, 0], v[:, 1] = 4.0, 2.0
    elif kind == "tiny":
        v = (v * np.float32(1e-42)).astype(np.float32)
    elif kind == "halves":
        v = (np.arange(300).reshape(6, 50) - 150).astype(np.float32) * 0.5 * np.float32(127 / 127)
        v[:, 0] = 127.0
    codes, scale = OI.quantize(v)
    for i in range(v.shape[0]):
        a = max(abs(Fraction(float(t))) for t in v[i])
        assert a > 0
        assert [_half_even(127 * Fraction(float(t)) / a) for t in v[i]] == codes[i].tolist()
        assert scale[i] == np.float32(float(a / 127)) or kind == "tiny"
    assert np.abs(codes.astype(int)).max() == 127


def test_zero_and_non_finite_rows():
    v = np.zeros((4, 8), np.float32)
    v[1, 3], v[2, 5], v[3, 0] = np.nan, -np.inf, 2.0
    codes, scale = OI.quantize(v)
    assert scale[0] == 0 and np.isnan(scale[1]) and np.isnan(scale[2]) and scale[3] == np.float32(2 / 127)
    assert not codes[:3].any() and codes[3].tolist() == [127] + [0] * 7


def test_rmsnorm_values_near_the_definition():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 96)).astype(np.float32)
    r = rng.standard_normal((5, 96)).astype(np.float32)
    g = (1 + 0.1 * rng.standard_normal(96)).astype(np.float32)
    codes, scale, h = OI.rmsnorm(x, g, 1e-6, r)
    h64 = x.astype(np.float64) + r
    y = h64 * g / np.sqrt((h64 ** 2).mean(axis=1, keepdims=True) + 1e-6)
    # a code is off by half a step of max|y| / 127
    step = np.abs(y).max(axis=1, keepdims=True) / 127
    assert np.all(np.abs(OI.dequantize(codes, scale) - y) <= 0.5001 * step)
    assert np.array_equal(h, x + r)
    codes, scale, _ = OI.rmsnorm(np.zeros((1, 8), np.float32), np.ones(8, np.float32), 0.0)
    assert not codes.any() and scale[0] == 0


def test_linear_sums_are_exact():
    rng = np.random.default_rng(5)
    w = rng.integers(-128, 128, (7, 640)).astype(np.int8)
    x = rng.integers(-128, 128, (3, 640)).astype(np.int8)
    one = np.ones(7, np.float32), np.ones(3, np.float32)
    want = (x.astype(np.int64) @ w.astype(np.int64).T).astype(np.float32)
    assert np.array_equal(OI.linear(w, one[0], x, one[1]), want)


def test_clip_factor_and_norm():
    g = [np.full(9, 2.0, np.float32), np.full((4, 4), -1.0, np.float32)]
    total, out = OC.clip(g, 1.0)
    assert total == math.sqrt(52)
    assert np.isclose(np.sqrt(sum((o.astype(np.float64) ** 2).sum() for o in out)), 1.0, rtol=1e-6)
    assert OC.factor(0.5, 1.0) == 1 and OC.factor(math.inf, 1.0) == 0 and np.isnan(OC.factor(math.nan, 1.0))
    assert OC.factor(math.inf, math.inf) == 1
    assert OC.norm([]) == 0.0
    assert math.isclose(OC.norm([np.full(4, 1e-30, np.float32)]), 2e-30, rel_tol=1e-6)
