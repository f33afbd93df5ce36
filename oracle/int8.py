"""8-bit rows, the norm that makes them and their product, in numpy.

For a row v with largest magnitude a: scale = fl32(a / 127), code = 127 v / a to
the nearest integer, ties to even, in exact arithmetic. float64 gives exactly
that for float32 rows: 127 v has 31 significant bits, and a quotient of such a
number by a 24-bit one that is no tie differs from every half-integer by more
than float64's rounding."""
import numpy as np


def quantize(v):
    """(codes int8, scale float32) of the rows of a float32 array."""
    v = np.asarray(v, dtype=np.float32).astype(np.float64)
    with np.errstate(invalid="ignore"):
        a = np.max(np.abs(v), axis=1, keepdims=True)  # NaN where a row has one
        bad = ~np.isfinite(a)
        live = ~bad & (a > 0)
        q = np.rint(np.where(live, v, 0.0) * 127.0 / np.where(live, a, 1.0))
    scale = np.where(bad, np.nan, np.where(live, a, 0.0) / 127.0).astype(np.float32)
    return q.astype(np.int8), scale[:, 0]


def dequantize(codes, scale):
    """float32 values: one float32 product each."""
    with np.errstate(over="ignore"):
        return codes.astype(np.float32) * scale[:, None].astype(np.float32)


def rmsnorm(x, gain, eps, residual=None):
    """(codes, scale, h): h = fl32(x + residual) in float32 (the caller rounds
    it to its type); the codes are those of fl32(h gain), the scale carries the
    norm's factor, with everything but the two float32 roundings in float64."""
    h = np.asarray(x, dtype=np.float32)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        v = h * np.asarray(gain, dtype=np.float32)
        codes, _ = quantize(v)
        h64 = h.astype(np.float64)
        mean = np.sum(h64 * h64, axis=1) / h.shape[1]
        a = np.max(np.abs(v.astype(np.float64)), axis=1)
        bad = ~(np.isfinite(a) & np.isfinite(mean))
        root = np.where(a > 0, np.sqrt(mean + float(np.float32(eps))), 1.0)
        scale = np.where(bad, np.nan, a / 127.0 / root).astype(np.float32)
    codes[bad] = 0
    return codes, scale, h


def linear(w, sw, x, sx):
    """float32 Y = (fl32(X W^T) sx) sw, the sums exact (whole numbers below 2^53)."""
    acc = x.astype(np.float64) @ w.astype(np.float64).T
    with np.errstate(over="ignore"):
        return (acc.astype(np.float32) * sx[:, None].astype(np.float32)) * sw[None, :].astype(np.float32)
