"""The gated feed-forward block's activation and product, and their gradient, in float64.

P = act(G) U with act(g) = g sigma(z): z = g (SiLU) or 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU, the tanh form, since
(1 + tanh t) / 2 = sigma(2 t)). act' = sigma + g sigma (1 - sigma) z'. An infinite gate counts as its limit."""
import math

import numpy as np

SILU, GELU = 0, 1
C = 2 * math.sqrt(2 / math.pi)


def _sigma(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def _z(g, act):
    """z(g) and g z'(g), whose product with sigma (1 - sigma) is the second term of act'."""
    if act == SILU:
        return g, g
    return C * (g + 0.044715 * g * g * g), C * (g + 3 * 0.044715 * g * g * g)


def value(g, act):
    g = np.asarray(g, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        v = g * _sigma(_z(g, act)[0])
    return np.where(np.isneginf(g), -0.0, v)


def slope(g, act):
    g = np.asarray(g, dtype=np.float64)
    t = np.clip(g, -200.0, 200.0)  # beyond, act' is within 1e-84 of its limits, 0 and 1
    z, tz = _z(t, act)
    s, r = _sigma(z), _sigma(-z)
    return np.where(np.isnan(g), np.nan, np.where(g < -200.0, 0.0, s + tz * s * r))


def fwd(g, u, act):
    with np.errstate(invalid="ignore", over="ignore"):
        return value(g, act) * np.asarray(u, dtype=np.float64)


def bwd(g, u, dp, act):
    """(dG, dU)."""
    u, dp = np.asarray(u, dtype=np.float64), np.asarray(dp, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        return dp * u * slope(g, act), dp * value(g, act)
