"""The gated product, its gradient and the 8-bit block in float32, against float64 at float32's own bounds.

Counted in half steps, u = 2^-24. sigma = r or e r with e = exp(-|z|) (2 u, and the error of z: none for SiLU, 4 u |z| for
the five roundings and constants of GELU's) and r = 1 / (1 + e) (2 u): relative 6 u + 4 u |z| sigma(-z), since an error of
e reaches sigma by the share of e in 1 + e; 1 - sigma the same with z turned round. act = g sigma and each product with it
are one more. act' = sigma + g z' sigma (1 - sigma): both relative errors and five roundings on the second term, one on the
sum. Below exp(-87.3) e is subnormal, 2^-149 off, and e r once more 2^-150: sigma is then up to 2 2^-149 off, act that
times |g|, and act' that times 1 + |g z'| (the second term's factor of sigma; 250 for GELU near g = -10)."""
import numpy as np
import pytest
import torch

import gated_cases as C
import test_gpu_int8_gated as I
from oracle import gated as OG

pytestmark = pytest.mark.gpu
U, LEAST = 2.0 ** -24, 2.0 ** -149


def sigma(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def parts(g, act):
    """z, g z' and the relative errors of sigma and 1 - sigma."""
    z, tz = OG._z(np.clip(g, -200.0, 200.0), act)
    wide = 4 * np.abs(z) if act == OG.GELU else 0 * z
    return z, tz, (6 + wide * sigma(-z)) * U, (6 + wide * sigma(z)) * U


def fwd_bound(g, u, act):
    _, _, rel, _ = parts(g, act)
    return np.abs(OG.fwd(g, u, act)) * (rel + 2 * U) * (1 + 2 ** -10) + (2 * np.abs(g * u) + 1) * LEAST


def bwd_bound(g, u, dp, act):
    z, tz, rel, rest = parts(g, act)
    s = sigma(z)
    second = np.abs(tz * s * sigma(-z))
    slope = s * rel + second * (rel + rest + 8 * U) + np.abs(OG.slope(g, act)) * U + 2 * (1 + np.abs(tz)) * LEAST
    dg, du = OG.bwd(g, u, dp, act)
    return (np.abs(dp * u) * slope * (1 + 2 ** -10) + np.abs(dg) * 3 * U + (1 + np.abs(dp)) * LEAST,
            np.abs(du) * (rel + 2 * U) * (1 + 2 ** -10) + (2 * np.abs(g * dp) + 1) * LEAST)


def compare(lib, gate, up, dp, act):
    """gate, up, dp: (m, n) float32 on the CPU."""
    y = torch.cat([gate, up], 1).cuda()
    g, u, d = C.f64(gate), C.f64(up), C.f64(dp)
    n = gate.shape[1]
    C.check(lib.gated_fwd(y, act), OG.fwd(g, u, act), fwd_bound(g, u, act), "P")
    dy = lib.gated_bwd(y, dp.cuda(), act)
    want, bound = OG.bwd(g, u, d, act), bwd_bound(g, u, d, act)
    C.check(dy[:, n:], want[1], bound[1], "dU")
    C.check(dy[:, :n], want[0], bound[0], "dG")


@pytest.mark.parametrize("act", C.ACTS)
def test_every_gate_of_a_range(gpu_lib, act):
    mags = torch.cat([torch.logspace(-30, 4, 2000, dtype=torch.float64), torch.linspace(0, 20, 4001, dtype=torch.float64),
                      torch.linspace(20, 130, 2201, dtype=torch.float64)])
    gate = torch.cat([mags, -mags]).float()[None]
    one = torch.ones_like(gate)
    compare(gpu_lib, gate, one, one, act)
    up, dp = C.normal(gate.shape, 1.0, 1).float(), C.normal(gate.shape, 1.0, 2).float()
    compare(gpu_lib, gate, up, dp, act)


@pytest.mark.parametrize("act", C.ACTS)
def test_gates_whose_sigma_is_next_to_nothing(gpu_lib, act):
    # SiLU: e^-88.7 is where e^88.7 leaves float32, e^-103.3 its least value; GELU reaches both at -9.6 and -10.3
    low, high = (-104.0, -85.0) if act == OG.SILU else (-10.5, -9.0)
    gate = torch.linspace(low, high, 1900, dtype=torch.float64).float()[None]
    big = torch.full_like(gate, 1e30)
    compare(gpu_lib, gate, big, big / 1e15, act)


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("m,n", [(1, 1), (3, 17), (37, 1001), (130, 264)])
def test_sizes(gpu_lib, m, n, act):
    y, dp = C.normal((m, 2 * n), 3.0, m + n).float(), C.normal((m, n), 1.0, 5).float()
    compare(gpu_lib, y[:, :n].contiguous(), y[:, n:].contiguous(), dp, act)


@pytest.mark.parametrize("act", C.ACTS)
def test_from_8_bit_rows(gpu_lib, act):
    m, n = 37, 1001
    q = gpu_lib.quantize_int8(C.normal((2 * m, n), 4.0, 3).float().cuda())
    y = gpu_lib.dequantize_int8(q, torch.float32).view(m, 2 * n)  # one rounded product, the kernel's own
    dp = C.normal((m, n), 1.0, 4).float().cuda()
    compare(gpu_lib, y[:, :n].contiguous().cpu(), y[:, n:].contiguous().cpu(), dp.cpu(), act)
    assert torch.equal(gpu_lib.gated_fwd(q, act, dtype=torch.float32), gpu_lib.gated_fwd(y, act))
    assert torch.equal(gpu_lib.gated_bwd(q, dp, act), gpu_lib.gated_bwd(y, dp, act))


# every kernel and several tiles
@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 7, 100), (16, 4095, 128), (1, 11008, 512), (40, 100, 1000), (300, 1030, 700), (1000, 2051, 192)])
def test_8_bit_block(gpu_lib, m, n, k, act):
    w, x, g, u = I.case(gpu_lib, m, n, k, m + n + k)
    p = gpu_lib.int8_linear_fwd_gated(w, x, act, torch.float32)
    # gate and up: the sum's rounding to float32 and the two scales'; |act'| < 1.13
    dg, du = 3 * U * np.abs(g), 3 * U * np.abs(u)
    with np.errstate(over="ignore"):
        bound = 1.14 * dg * np.abs(u) + np.abs(OG.value(g, act)) * du * 1.01 + fwd_bound(g, u, act)
    C.check(p, OG.fwd(g, u, act), bound, "P")
