"""The least workspace of the gated block and of the backward from 8-bit rows (no GPU): what the calls take without the
restored weight. Fake aligned addresses stand in; calls are refused, or end at their first launch, no device being there."""
import ctypes
import itertools

import pytest
import torch

from bit_nf4_quantized_18_amd import binding as B

G = 1 << 36
AT = {name: (i + 1) * G for i, name in enumerate(
    ("codes", "sc", "gs", "x", "a", "b", "y", "p", "h", "ws", "dy", "dx", "da", "db", "xs"))}
SIZES = list(itertools.product([1, 16, 17, 40, 333, 2048], [512, 1024, 22016], [64, 1088, 4096], [0, 5, 16, 64]))


def restored(n, k):
    return (2 * n * k + 255) // 256 * 256


def test_sizes():
    some = 0
    for m, n, k, r in SIZES:
        full, least = B.gated_workspace_bytes(m, n, k, r), B.gated_workspace_bytes(m, n, k, r, restored=False)
        assert full - least in (0, restored(n, k)) and 0 <= least < 1 << 28, (m, n, k, r)
        some += full > least
        full, least = B.x8_workspace_bytes(m, n, k, 1, r), B.x8_workspace_bytes(m, n, k, 1, r, restored=False)
        assert full - least in (0, restored(n, k)) and 0 <= least < 1 << 28, (m, n, k, r)
        some += full > least
    assert some > 50
    for bad in ((0, 512, 64), (10, 0, 64), (10, 512, -1), (1 << 40, 512, 64)):
        assert B.gated_workspace_bytes(*bad, 16, restored=False) == 0 and B.x8_workspace_bytes(*bad, 1, 16, restored=False) == 0
    assert B.gated_workspace_bytes(40, 512, 64, 65, restored=False) == 0 and B.gated_workspace_bytes(40, 512, 64, 1 << 30, restored=False) == 0
    assert B.x8_workspace_bytes(40, 512, 64, 5, 16, restored=False) == 0 and B.x8_workspace_bytes(40, 512, 64, 4, 1 << 30, restored=False) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none")
def test_calls_take_it():
    lib = B.load()
    for m, n, k, r in SIZES:
        w = B.NF4WeightC(n, k, AT["codes"], AT["sc"], AT["gs"], None, 1, 0)
        least = B.gated_workspace_bytes(m, n, k, r, restored=False)
        block = lambda size: lib.qlora_linear_fwd_gated(ctypes.byref(w), AT["x"], m, AT["a"], AT["b"], r, 32.0, 0, AT["y"],  # noqa: E731
                                                        AT["p"], AT["h"], AT["ws"] if size else None, size, None)
        assert block(least) == -6 and (least == 0 or block(least - 1) == -5), (m, n, k, r)
        least = B.x8_workspace_bytes(m, n, k, 1, r, restored=False)
        for dx in (AT["dx"], None):
            back = lambda size: lib.qlora_linear_bwd_x8(ctypes.byref(w), AT["x"], k, AT["xs"], AT["dy"], m, AT["a"], AT["b"],  # noqa: E731
                                                        r, 32.0, AT["h"], dx, AT["da"], AT["db"], AT["ws"] if size else None, size, None)
            want = -6 if dx or r else 0  # neither gradient: nothing to do
            assert back(least) == want and (least == 0 or want == 0 or back(least - 1) == -5), (m, n, k, r, dx)


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none")
def test_memory_that_no_output_needs_may_hold_others():
    # without dX the restored weight's place is not used: an output may lie there
    m, n, k, r = 333, 1024, 1088, 16
    w = B.NF4WeightC(n, k, AT["codes"], AT["sc"], AT["gs"], None, 1, 0)
    full, least = B.x8_workspace_bytes(m, n, k, 1, r), B.x8_workspace_bytes(m, n, k, 1, r, restored=False)
    assert full - least == restored(n, k)

    def back(dx, da):
        return B.load().qlora_linear_bwd_x8(ctypes.byref(w), AT["x"], k, AT["xs"], AT["dy"], m, AT["a"], AT["b"], r, 32.0,
                                            AT["h"], dx, da, AT["db"], AT["ws"], full, None)

    assert back(AT["dx"], AT["ws"] + least) == -4 and back(None, AT["ws"] + least) == -6
    assert back(None, AT["ws"] + least - 256) == -4
