"""Shared helpers of the gated-block and 8-bit checkpoint tests: seeded inputs, float64 results and error bounds.

Bounds count roundings: half a step eps / 2 |value| where a result is rounded to its type, 2^-24 a term for float32
sums of n terms (n 2^-24 sum |terms|), 2^-16 relative for the 16-bit kernels' sigma (2^-21 (1 + |z|), |z| < 89 where it
is not 0) and at most 1.13 for |act'|."""
import numpy as np
import torch

from oracle import gated as OG

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = [OG.SILU, OG.GELU]
F32 = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the smallest step of a type, for results under its normal range; float32 kernels may flush these."""
    info = torch.finfo(t)
    return float(info.tiny) if t == torch.float32 else float(info.smallest_normal) * info.eps / 2


def normal(shape, std, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * std)


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, want, tol, name):
    """|got - want| <= tol element by element; NaN and infinities where want has them."""
    got = f64(got)
    fine = np.isfinite(want)
    assert got.shape == want.shape, name
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{name}: NaN elsewhere than expected"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{name}: infinities differ"
    off = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, want.shape)[fine]
    worst = off.max() if off.size else 0.0
    assert worst <= 0, f"{name}: {worst:.3g} over its bound"


def fwd_bound(g, u, act, t, dg=0.0, du=0.0):
    """For P from gates and ups that are themselves dg and du off."""
    p = OG.fwd(g, u, act)
    with np.errstate(invalid="ignore", over="ignore"):
        wide = 1.13 * dg * (np.abs(u) + du) + np.abs(OG.value(g, act)) * du
        return np.abs(p) * (half_step(t) + 2.0 ** -16) * (1 + 2 ** -8) + 1.01 * wide + tiny(t) + 1e-36 * np.abs(g * u)


def bwd_bound(g, u, dp, act, t):
    """(for dG, for dU). sigma's relative error 2^-22 where it is near 1 meets a factor |g z'| below 51 there, in
    1 - sigma: 2^-16 |dP U| absolutely, doubled."""
    dg, du = OG.bwd(g, u, dp, act)
    with np.errstate(invalid="ignore", over="ignore"):
        rel = half_step(t) + 2.0 ** -16
        return (np.abs(dg) * rel + np.abs(dp * u) * 2.0 ** -15 + tiny(t),
                np.abs(du) * rel + tiny(t) + 1e-36 * np.abs(g * dp))
