"""Pins of the gated block's oracle: torch's own activations, central differences, limits, a literal product."""
import math

import numpy as np
import torch

from oracle import gated as O

G = np.concatenate([np.linspace(-30, 30, 4001), -np.logspace(-9, 2.5, 400), np.logspace(-9, 2.5, 400)])


def test_values_are_torchs():
    t = torch.from_numpy(G)
    for act, f in ((O.SILU, torch.nn.functional.silu), (O.GELU, lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
        # torch's tanh form cancels in 1 + tanh for negative gates: 2^-52 of |g| / 2
        assert (np.abs(O.value(G, act) - f(t).numpy()) <= 1e-15 * (1 + np.abs(G))).all()


def test_slopes_are_autograds_and_differences():
    for act, f in ((O.SILU, torch.nn.functional.silu), (O.GELU, lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
        t = torch.from_numpy(G).requires_grad_()
        f(t).sum().backward()
        assert (np.abs(O.slope(G, act) - t.grad.numpy()) <= 1e-13 * (1 + np.abs(G))).all()
        h = 2.0 ** -14
        diff = (O.value(G + h, act) - O.value(G - h, act)) / (2 * h)
        # h^2 / 6 |act'''| with |act'''| < 3, and 2^-52 of |g| over h
        assert (np.abs(O.slope(G, act) - diff) <= 0.5 * h * h + 2.0 ** -51 * (1 + np.abs(G)) / h).all()


def test_limits():
    inf = math.inf
    for act in (O.SILU, O.GELU):
        assert O.value(-inf, act) == 0 and O.value(inf, act) == inf and np.isnan(O.value(math.nan, act))
        assert O.slope(-inf, act) == 0 and O.slope(inf, act) == 1 and np.isnan(O.slope(math.nan, act))
        assert O.slope(-1e30, act) == 0 and O.slope(1e30, act) == 1 and O.value(1e30, act) == 1e30


def test_a_literal_product():
    g, u, dp = 0.7, -1.3, 2.1
    s = 1 / (1 + math.exp(-g))
    assert O.fwd(g, u, O.SILU) == np.float64(g * s) * u
    dg, du = O.bwd(g, u, dp, O.SILU)
    assert math.isclose(dg, dp * u * (s + g * s * (1 - s)), rel_tol=1e-15) and math.isclose(du, dp * g * s, rel_tol=1e-15)
