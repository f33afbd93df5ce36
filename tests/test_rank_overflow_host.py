"""Ranks whose product with the number of parts leaves 32 bits (no GPU): sizes are 0 and the calls refuse them.

Fake aligned addresses, far apart, stand in; every call is refused before a launch."""
import ctypes

import pytest

from bit_nf4_quantized_18_amd import binding as B

G = 1 << 32
AT = {name: (i + 1) * G for i, name in enumerate(
    ("codes", "sc", "gs", "x", "a", "b", "y", "p", "h", "ws", "dy", "dx", "da", "db", "xs"))}
# times 2, 3 or 4 these wrap to a rank that would pass, to 0 or below it
RANKS = [(1 << 30) - 1, 1 << 30, (1 << 30) + 16, (1 << 29) + 16, (1 << 31) - 16, (1 << 31) - 1, 1431655766, 129]
MANY = 1 << 62  # bytes of workspace


def weight():
    return B.NF4WeightC(1024, 128, AT["codes"], AT["sc"], AT["gs"], None, 1, 0)


@pytest.mark.parametrize("r", RANKS)
def test_workspace_queries(r):
    assert B.gated_workspace_bytes(300, 512, 64, r) == 0 and B.gated_workspace_bytes(1, 512, 64, r) == 0
    for g in (1, 2, 3, 4):
        assert B.x8_workspace_bytes(300, 512, 64, g, r) == 0, g
        assert B.grouped_workspace_bytes(300, 512, 64, g, r) == 0, g


@pytest.mark.parametrize("dx", [None, AT["dx"]])
@pytest.mark.parametrize("f16", ["", "_f16"])
@pytest.mark.parametrize("r", RANKS)
def test_grouped_calls(r, f16, dx):
    lib, w = B.load(), weight()
    for g in (2, 4):
        parts = B._parts([1024 // g] * g)
        lead = (ctypes.byref(w), g, parts)
        tail = (AT["a"], AT["b"], r, 32.0, AT["h"], dx, AT["da"], AT["db"], AT["ws"], MANY, None)
        x8 = getattr(lib, "qlora_linear_bwd_grouped_x8" + f16)
        assert x8(*lead, AT["x"], 128, AT["xs"], AT["dy"], 40, *tail) == -4, g
        bwd = getattr(lib, "qlora_linear_bwd_grouped" + f16)
        assert bwd(*lead, AT["x"], AT["dy"], 40, *tail) == -4, g
        fwd = getattr(lib, "qlora_linear_fwd_grouped" + f16)
        assert fwd(*lead, AT["x"], 40, AT["a"], AT["b"], r, 32.0, AT["y"], AT["h"], AT["ws"], MANY, None) == -4, g


@pytest.mark.parametrize("r", RANKS)
def test_block(r):
    w = weight()
    call = B.load().qlora_linear_fwd_gated
    assert call(ctypes.byref(w), AT["x"], 40, AT["a"], AT["b"], r, 32.0, 0, AT["y"], AT["p"], AT["h"], AT["ws"], MANY, None) == -4
