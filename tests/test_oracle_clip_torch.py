"""The clipping oracle against torch's clip_grad_norm_ (CPU): the same values,
NaN and infinite norms included, but for an infinite max_norm beside a norm
that is not finite."""
import math

import numpy as np
import pytest
import torch

from oracle import clip as OC


def _grads(bad):
    rng = np.random.default_rng(6)
    g = [rng.standard_normal(s).astype(np.float32) for s in (50, 7, 300)]
    if bad is not None:
        g[1][3] = bad
    return g


def _torch_clip(g, max_norm):
    p = [torch.nn.Parameter(torch.zeros(v.shape)) for v in g]
    for q, v in zip(p, g):
        q.grad = torch.from_numpy(v.copy())
    torch.nn.utils.clip_grad_norm_(p, max_norm)
    return [q.grad.numpy() for q in p]


@pytest.mark.parametrize("bad", [None, math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e3, 3e38])
def test_same_values(bad, max_norm):
    g = _grads(bad)
    _, mine = OC.clip(g, max_norm)
    for a, b in zip(mine, _torch_clip(g, max_norm)):
        assert np.array_equal(np.isnan(a), np.isnan(b))
        # torch's norm is summed in float32: 357 squares, 2^-24 each at most, and three roundings behind
        assert np.allclose(a, b, rtol=360 * 2.0 ** -24, atol=0, equal_nan=True)


@pytest.mark.parametrize("bad", [None, math.nan, math.inf])
def test_infinite_max_norm(bad):
    g = _grads(bad)
    _, mine = OC.clip(g, math.inf)
    assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(mine, g))
    theirs = _torch_clip(g, math.inf)
    if bad is None:
        assert all(np.array_equal(a, b) for a, b in zip(theirs, g))
    else:
        assert all(np.isnan(b).all() for b in theirs)
