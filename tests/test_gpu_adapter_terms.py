"""The adapter's part of the gated block and of dX from 8-bit rows holds H and dH in 32 bits, at every number of tokens.

The weight is zero and the slots come in pairs that nearly cancel, so a rounding of s H (or dH) to 16 bits, 2^-9 (2^-12) of
each term, would stand far above the bounds here: n 2^-24 of the terms for a float32 sum of n, and the result's own
rounding, 2^-4 smaller than the terms."""
import numpy as np
import pytest
import torch

import gated_cases as C
from oracle import gated as OG

pytestmark = pytest.mark.gpu


def pairs(rows, r, along, t, seed):
    """(rows, r) positive values whose columns 2 p and 2 p + 1 differ by up to 2^-4 of them, and (r, along) factors of
    opposite sign for the two; the last column of an odd r meets zeros."""
    rng = np.random.default_rng(seed)
    near = rng.uniform(0.5, 1.5, (rows, r))
    near[:, 1::2] = near[:, : r - r % 2: 2] * (1 + rng.uniform(-1, 1, (rows, r // 2)) / 16)
    far = rng.standard_normal((r, along))
    far[1::2] = -far[: r - r % 2: 2]
    if r % 2:
        far[-1] = 0
    return torch.from_numpy(near).to(t), torch.from_numpy(far).to(t)


def block(lib, m, half, k, r, t, seed, top):
    """A block whose H has values near `top` / s."""
    w = lib.quantize(torch.zeros(2 * half, k, device="cuda"))
    x = torch.from_numpy(np.random.default_rng(seed).uniform(0.5, 1.5, (m, k))).to(t)
    a, b = zip(*(pairs(k, r, half, t, seed + l) for l in (1, 2)))
    a = torch.cat([v.t() for v in a]).contiguous()
    b = torch.cat([v.t() for v in b])
    s = top / k
    b = (b.double() * 2.0 ** np.round(np.log2(16 / top))).to(t)  # Y of unit size
    return w, x.cuda(), a.cuda(), b.contiguous().cuda(), s * r


def block_expected(x, a, b, alpha, half):
    r, k = b.shape[1], x.shape[1]
    s = np.float64(np.float32(alpha / r))
    x64, a64, b64 = (v.cpu().double().numpy() for v in (x, a, b))
    v, off = np.zeros((x.shape[0], 2 * half)), np.zeros((x.shape[0], 2 * half))
    for l in range(2):
        h = x64 @ a64[l * r:(l + 1) * r].T  # of positive terms
        bt = b64[l * half:(l + 1) * half].T
        v[:, l * half:(l + 1) * half] = s * (h @ bt)
        # H in float32, s, and at most six products a slot, float32 sums of exact products
        off[:, l * half:(l + 1) * half] = s * (h @ np.abs(bt)) * ((k + 6 * r + 3) * C.F32)
    return v, off


def check_block(lib, m, half, k, r, kind, act, top, ws):
    t = C.TYPES[kind]
    w, x, a, b, alpha = block(lib, m, half, k, r, t, m + r, top)
    p, y, h = lib.linear_fwd_gated(w, x, a, b, alpha, act, ws=ws)
    v, off = block_expected(x, a, b, alpha, half)
    C.check(y, v, np.abs(v) * C.half_step(t) * (1 + 2 ** -7) + off * 1.01 + C.tiny(t), "Y")
    g, u = v[:, :half], v[:, half:]
    C.check(p, OG.fwd(g, u, act), C.fwd_bound(g, u, act, t, off[:, :half], off[:, half:]), "P")


# fp16's largest value is 65504: s H = 5e5 has none of its own there
TOPS = [("bf16", 64.0), ("fp16", 64.0), ("fp16", 5e5)]


@pytest.mark.parametrize("kind,top", TOPS)
@pytest.mark.parametrize("r", [2, 5, 16, 64])
@pytest.mark.parametrize("m", [5, 40, 300])
def test_block(gpu_lib, m, r, kind, top):
    check_block(gpu_lib, m, 512, 320, r, kind, r % 2, top, None)


@pytest.mark.parametrize("kind,top", TOPS)
@pytest.mark.parametrize("r", [2, 5, 16, 64])
def test_block_restored_as_it_is_multiplied(gpu_lib, r, kind, top):
    m, half, k = 300, 512, 320
    without = gpu_lib.gated_workspace_bytes(m, 2 * half, k, r) - 2 * 2 * half * k
    ws = torch.empty(without, dtype=torch.uint8, device="cuda")
    check_block(gpu_lib, m, half, k, r, kind, OG.SILU, top, ws)


def backward(lib, m, n, k, parts, r, t, seed, top):
    """A backward pass whose dH has values near `top`."""
    rows = n // parts
    w = lib.quantize(torch.zeros(n, k, device="cuda"))
    dy = torch.from_numpy(np.random.default_rng(seed).uniform(0.5, 1.5, (m, n))).to(t)
    b, a = zip(*(pairs(rows, r, k, t, seed + 1 + l) for l in range(parts)))
    scale = 2.0 ** np.round(np.log2(16 / top))
    a = (torch.cat(a).double() * scale).to(t)
    x = lib.quantize_int8(C.normal((m, k), 1.0, seed + 9).to(t).cuda())
    h = C.normal((m, parts * r), 1.0, seed + 10).float().cuda()
    return w, x, dy.cuda(), h, a.contiguous().cuda(), torch.cat(b).contiguous().cuda(), top / rows * r


def check_backward(lib, m, n, k, parts, r, kind, top, ws=None):
    t = C.TYPES[kind]
    w, x, dy, h, a, b, alpha = backward(lib, m, n, k, parts, r, t, m + r, top)
    if parts == 1:
        dx = lib.linear_bwd(w, x, dy, a, b, alpha, h=h, ws=ws)[0]
    else:
        dx = lib.linear_bwd_grouped(w, [n // parts] * parts, x, dy, a, b, alpha, h=h, ws=ws)[0]
    s = np.float64(np.float32(alpha / r))
    dy64, a64, b64 = (v.cpu().double().numpy() for v in (dy, a, b))
    v, off = np.zeros((m, k)), np.zeros((m, k))
    for l in range(parts):
        cols, slots = slice(l * (n // parts), (l + 1) * (n // parts)), slice(l * r, (l + 1) * r)
        dh = s * (dy64[:, cols] @ b64[cols])  # of positive terms
        v += dh @ a64[slots]
        off += (dh @ np.abs(a64[slots])) * ((n // parts + 6 * parts * r + 3) * C.F32)
    C.check(dx, v, np.abs(v) * C.half_step(t) * (1 + 2 ** -7) + off * 1.01 + C.tiny(t), "dX")


@pytest.mark.parametrize("kind,top", TOPS)
@pytest.mark.parametrize("r", [2, 5, 16, 64])
@pytest.mark.parametrize("m", [5, 300])
def test_backward(gpu_lib, m, r, kind, top):
    check_backward(gpu_lib, m, 272, 320, 1, r, kind, top)


@pytest.mark.parametrize("kind,top", TOPS)
@pytest.mark.parametrize("parts,r", [(2, 16), (3, 16), (2, 64)])
def test_backward_grouped(gpu_lib, parts, r, kind, top):
    check_backward(gpu_lib, 77, 256 * parts, 320, parts, r, kind, top)


@pytest.mark.parametrize("kind,top", TOPS)
def test_backward_of_many_weight_rows(gpu_lib, kind, top):
    check_backward(gpu_lib, 40, 4112, 320, 1, 2, kind, top)  # dH in launches of its own


@pytest.mark.parametrize("kind,top", TOPS)
@pytest.mark.parametrize("n,parts,r", [(272, 1, 2), (272, 1, 5), (512, 2, 16)])
def test_backward_restored_as_it_is_multiplied(gpu_lib, n, parts, r, kind, top):
    m, k = 300, 320
    without = gpu_lib.x8_workspace_bytes(m, n, k, parts, r) - 2 * n * k
    ws = torch.empty(without, dtype=torch.uint8, device="cuda")
    check_backward(gpu_lib, m, n, k, parts, r, kind, top, ws)
