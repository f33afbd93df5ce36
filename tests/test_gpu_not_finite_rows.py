"""Tokens, adapter rows and gradients that are not finite, in the gated block and the backward from 8-bit rows: they come
out as NaN or infinity where the header says, and every other output is bit for bit what it is without them. Where n is no
multiple of 64 the fused product reads a row of dY on into the next one against zeros, so the token in front of one that
is not finite may get NaN as well (the header's rule for all linear calls)."""
import pytest
import torch

import gated_cases as C
import test_gpu_linear_gated as L
import test_gpu_linear_x8 as X

pytestmark = pytest.mark.gpu
BAD = [float("inf"), float("-inf"), float("nan")]


def same(got, want, rest):
    """Equal where `rest`, nothing finite elsewhere."""
    assert torch.equal(got[rest], want[rest])
    assert not torch.isfinite(got[~rest]).any()


def workspace(full, least, small):
    return torch.empty(least, dtype=torch.uint8, device="cuda") if small and least else None


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [5, 16, 300])
def test_block(gpu_lib, m, kind, small):
    half, k, r, t = 512, 320, 16, C.TYPES[kind]
    w, x, a, b, alpha = L.layer(gpu_lib, m, half, k, r, t, 5)
    least = gpu_lib.gated_workspace_bytes(m, 2 * half, k, r, restored=False)
    call = lambda *v: gpu_lib.linear_fwd_gated(w, *v, alpha, ws=workspace(0, least, small))  # noqa: E731
    p, y, h = call(x, a, b)
    for bad in BAD:
        # a token: its own rows
        x2 = x.clone()
        x2[3, 100] = bad
        rest = torch.ones(m, dtype=torch.bool, device="cuda")
        rest[3] = False
        p2, y2, h2 = call(x2, a, b)
        assert torch.equal(p2[rest], p[rest]) and torch.equal(y2[rest], y[rest]) and torch.equal(h2[rest], h[rest])
        assert not torch.isfinite(y2[3]).any() and not torch.isfinite(h2[3]).any()
        # a row of B, up's 7: its own weight row
        b2 = b.clone()
        b2[half + 7, 2] = bad
        p2, y2, h2 = call(x, a, b2)
        keep = torch.ones(2 * half, dtype=torch.bool, device="cuda")
        keep[half + 7] = False
        assert torch.equal(y2[:, keep], y[:, keep]) and torch.equal(p2[:, keep[half:]], p[:, keep[half:]]) and torch.equal(h2, h)
        assert not torch.isfinite(y2[:, half + 7]).any() and not torch.isfinite(p2[:, 7]).any()
        # a row of A: its slot of H
        a2 = a.clone()
        a2[r + 1, 64] = bad
        h2 = call(x, a2, b)[2]
        slots = torch.ones(2 * r, dtype=torch.bool, device="cuda")
        slots[r + 1] = False
        assert torch.equal(h2[:, slots], h[:, slots]) and not torch.isfinite(h2[:, r + 1]).any()


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("parts,n", [(1, 272), (2, 512), (1, 4112)])
@pytest.mark.parametrize("m", [5, 300])
def test_backward(gpu_lib, m, parts, n, kind, small):
    k, r, t = 320, 16, C.TYPES[kind]
    w, x, dy, h, a, b, alpha = X.layer(gpu_lib, m, n, k, parts, r, t, 6)
    least = gpu_lib.x8_workspace_bytes(m, n, k, parts, r, restored=False)
    call = lambda *v: X.call(gpu_lib, w, x, *v, alpha, parts, ws=workspace(0, least, small))  # noqa: E731
    dx, da, db = call(dy, h, a, b)
    rows = torch.ones(m, dtype=torch.bool, device="cuda")
    rows[2] = False
    for bad in BAD:
        # an element of dY: its token's dX, its row of dB, all of dA
        dy2 = dy.clone()
        dy2[2, 9] = bad
        dx2, da2, db2 = call(dy2, h, a, b)
        cols = torch.ones(n, dtype=torch.bool, device="cuda")
        cols[9] = False
        if n % 64:
            dx2[1] = dx[1]
        same(dx2, dx, rows), same(db2, db, cols)
        assert not torch.isfinite(da2).any()
        # an element of H: its slot of dB
        h2 = h.clone()
        h2[2, 3] = bad
        dx2, da2, db2 = call(dy, h2, a, b)
        slot = torch.ones(n, r, dtype=torch.bool, device="cuda")
        slot[: n // parts, 3] = False
        assert torch.equal(dx2, dx) and torch.equal(da2, da)
        same(db2, db, slot)
        # a row of B: its slot of dH, so of dA, and dX
        b2 = b.clone()
        b2[n - 1, 4] = bad
        dx2, da2, db2 = call(dy, h, a, b2)
        slots = torch.ones(parts * r, dtype=torch.bool, device="cuda")
        slots[(parts - 1) * r + 4] = False
        same(da2, da, slots)
        assert torch.equal(db2, db) and not torch.isfinite(dx2).any()
        # a column of A: its column of dX
        a2 = a.clone()
        a2[1, 77] = bad
        dx2, da2, db2 = call(dy, h, a2, b)
        inputs = torch.ones(k, dtype=torch.bool, device="cuda")
        inputs[77] = False
        assert torch.equal(da2, da) and torch.equal(db2, db)
        assert torch.equal(dx2[:, inputs], dx[:, inputs]) and not torch.isfinite(dx2[:, 77]).any()
