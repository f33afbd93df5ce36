"""The global norm of a list of gradients and clipping by it, in numpy."""
import math

import numpy as np


def norm(grads):
    """sqrt of the sum of all squares (float64; the sum correctly rounded)."""
    flat = [np.asarray(g).astype(np.float64).reshape(-1) for g in grads]
    if not all(np.isfinite(f).all() for f in flat):
        return math.nan if any(np.isnan(f).any() for f in flat) else math.inf
    return math.sqrt(math.fsum(float(v) * float(v) for f in flat for v in f))


def factor(total, max_norm):
    """fl32(min(1, max_norm / (norm + 1e-6))); 1 for an infinite max_norm, whatever the norm."""
    if math.isinf(max_norm):
        return np.float32(1.0)
    if math.isnan(total):
        return np.float32(np.nan)
    return np.float32(min(1.0, float(np.float32(max_norm)) / (total + 1e-6)))


def clip(grads, max_norm):
    """(norm, float32 clipped gradients)."""
    total = norm(grads)
    f = factor(total, max_norm)
    with np.errstate(invalid="ignore"):
        return total, [np.asarray(g, dtype=np.float32) * f for g in grads]
