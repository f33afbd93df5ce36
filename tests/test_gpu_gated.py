"""The gated block's product and gradient, element by element, against float64."""
import numpy as np
import pytest
import torch

import gated_cases as C
from oracle import gated as OG

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (2, 7), (3, 17), (5, 64), (37, 1001), (2, 5001), (130, 264), (1, 11008)]


def inputs(m, n, t, seed):
    y = C.normal((m, 2 * n), 3.0, seed).to(t)
    dp = C.normal((m, n), 1.0, seed + 1).to(t)
    return y, dp


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("kind", list(C.TYPES))
@pytest.mark.parametrize("m,n", SHAPES)
def test_product_and_gradient(gpu_lib, m, n, kind, act):
    t = C.TYPES[kind]
    y, dp = inputs(m, n, t, m * 7 + n)
    p = gpu_lib.gated_fwd(y.cuda(), act)
    dy = gpu_lib.gated_bwd(y.cuda(), dp.cuda(), act)
    assert p.dtype is t and dy.dtype is t
    g, u, d = C.f64(y[:, :n]), C.f64(y[:, n:]), C.f64(dp)
    C.check(p, OG.fwd(g, u, act), C.fwd_bound(g, u, act, t), "P")
    want, bound = OG.bwd(g, u, d, act), C.bwd_bound(g, u, d, act, t)
    C.check(dy[:, :n], want[0], bound[0], "dG")
    C.check(dy[:, n:], want[1], bound[1], "dU")


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("kind", list(C.TYPES))
@pytest.mark.parametrize("m,n", SHAPES)
def test_from_8_bit_rows(gpu_lib, m, n, kind, act):
    t = C.TYPES[kind]
    y, dp = inputs(m, n, t, m * 5 + n)
    q = gpu_lib.quantize_int8(y.cuda().view(2 * m, n))
    p = gpu_lib.gated_fwd(q, act, dtype=t)
    dy = gpu_lib.gated_bwd(q, dp.cuda(), act)
    v = (C.f64(q.codes)[:, :n] * C.f64(q.scale)[:, None]).reshape(m, 2 * n)
    g, u, d = v[:, :n], v[:, n:], C.f64(dp)
    # gate and up are products rounded to float32: one rounding each
    bound = C.fwd_bound(g, u, act, t, np.abs(g) * C.F32, np.abs(u) * C.F32)
    C.check(p, OG.fwd(g, u, act), bound, "P")
    want, bound = OG.bwd(g, u, d, act), C.bwd_bound(g, u, d, act, t)
    C.check(dy[:, :n], want[0], bound[0], "dG")
    C.check(dy[:, n:], want[1], bound[1], "dU")


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("kind", list(C.TYPES))
def test_every_gate_of_a_range(gpu_lib, kind, act):
    t = C.TYPES[kind]
    top = 60000.0 if kind == "fp16" else 1e30
    mags = torch.cat([torch.logspace(-8, np.log10(top), 700, dtype=torch.float64), torch.linspace(0, 120, 1501, dtype=torch.float64)])
    gate = torch.cat([mags, -mags]).to(t)
    up = torch.ones_like(gate)
    y = torch.cat([gate, up])[None]
    dp = torch.ones(1, gate.numel(), dtype=t)
    p, dy = gpu_lib.gated_fwd(y.cuda(), act), gpu_lib.gated_bwd(y.cuda(), dp.cuda(), act)
    g, u, d = C.f64(gate)[None], C.f64(up)[None], C.f64(dp)
    C.check(p, OG.fwd(g, u, act), C.fwd_bound(g, u, act, t), "P")
    want, bound = OG.bwd(g, u, d, act), C.bwd_bound(g, u, d, act, t)
    n = gate.numel()
    C.check(dy[:, :n], want[0], bound[0], "dG")
    C.check(dy[:, n:], want[1], bound[1], "dU")


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("kind", list(C.TYPES))
def test_values_that_are_not_finite(gpu_lib, kind, act):
    t = C.TYPES[kind]
    inf, nan = float("inf"), float("nan")
    gate = torch.tensor([inf, -inf, nan, 1.0, 1.0, 0.0, -0.0, -inf, 2.0], dtype=t)
    up = torch.tensor([2.0, 2.0, 2.0, inf, nan, 3.0, 3.0, -1.0, -inf], dtype=t)
    dp = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, nan], dtype=t)
    y = torch.cat([gate, up])[None].cuda()
    p, dy = gpu_lib.gated_fwd(y, act), gpu_lib.gated_bwd(y, dp[None].cuda(), act)
    n = gate.numel()
    p, dg, du = C.f64(p)[0], C.f64(dy)[0, :n], C.f64(dy)[0, n:]
    assert p[0] == inf and p[1] == 0 and np.isnan(p[2]) and p[3] == inf and np.isnan(p[4]) and p[5] == 0 and p[8] == -inf
    assert dg[0] == 2 and dg[1] == 0 and np.isnan(dg[2]) and dg[3] == inf and np.isnan(dg[4]) and dg[5] == 1.5
    assert du[0] == inf and du[1] == 0 and np.isnan(du[2]) and du[5] == 0 and du[7] == 0 and np.isnan(du[8])


def test_a_row_that_quantized_to_nan(gpu_lib):
    y = C.normal((3, 2 * 40), 1.0, 5).to(torch.bfloat16)
    y[1, 3] = float("nan")  # token 1's gate: its row's scale becomes NaN
    q = gpu_lib.quantize_int8(y.cuda().view(6, 40))
    dy = gpu_lib.gated_bwd(q, torch.ones(3, 40, dtype=torch.bfloat16, device="cuda"))
    p = gpu_lib.gated_fwd(q)
    assert torch.isnan(p[1]).all() and torch.isnan(dy[1]).all()
    assert torch.isfinite(p[[0, 2]]).all() and torch.isfinite(dy[[0, 2]]).all()


def test_gradient_against_differences(gpu_lib):
    m, n, h = 4, 33, 2.0 ** -7
    for act in C.ACTS:
        y = C.normal((m, 2 * n), 2.0, 3 + act).float()
        dp = C.normal((m, n), 1.0, 9).float()
        dy = C.f64(gpu_lib.gated_bwd(y.cuda(), dp.cuda(), act))
        for half, cols in ((0, slice(0, n)), (1, slice(n, 2 * n))):
            up, down = y.clone(), y.clone()
            up[:, cols] += h
            down[:, cols] -= h
            step = C.f64(up[:, cols]) - C.f64(down[:, cols])
            diff = (C.f64(gpu_lib.gated_fwd(up.cuda(), act)) - C.f64(gpu_lib.gated_fwd(down.cuda(), act))) * C.f64(dp) / step
            # a central difference is h^2 / 6 |act'''| off, |act'''| < 3 for both, and its float32
            # values 2^-22 of P each over the step; U's part is linear
            p = np.abs(C.f64(gpu_lib.gated_fwd(y.cuda(), act))) + 1
            tol = np.abs(C.f64(dp)) * (0.5 * h * h * (np.abs(C.f64(y[:, n:])) if half == 0 else 0) + 2 * p * 2.0 ** -20 / h)
            assert (np.abs(diff - dy[:, cols]) <= tol + 1e-6).all(), (act, half)


def test_in_place_and_preallocated(gpu_lib):
    m, n = 19, 301
    y, dp = inputs(m, n, torch.float16, 1)
    y, dp = y.cuda(), dp.cuda()
    want_p, want = gpu_lib.gated_fwd(y), gpu_lib.gated_bwd(y, dp)
    room = torch.full((m * 2 * n + 64,), 7.0, dtype=torch.float16, device="cuda")
    out = room[: m * n].view(m, n)
    assert gpu_lib.gated_fwd(y, out=out) is out and torch.equal(out, want_p)
    assert (room[m * n:] == 7.0).all()  # nothing behind the last row
    both = room[: 2 * m * n].view(m, 2 * n)
    assert gpu_lib.gated_bwd(y, dp, out=both) is both and torch.equal(both, want)
    assert (room[2 * m * n:] == 7.0).all()
    assert gpu_lib.gated_bwd(y, dp, out=y) is y and torch.equal(y, want)


def test_no_tokens(gpu_lib):
    y = torch.empty(0, 20, dtype=torch.bfloat16, device="cuda")
    dp = torch.empty(0, 10, dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.gated_fwd(y).shape == (0, 10) and gpu_lib.gated_bwd(y, dp).shape == (0, 20)


def test_captured_with_eager_calls_between(gpu_lib):
    m, n = 33, 520
    y, dp = (v.cuda() for v in inputs(m, n, torch.bfloat16, 2))
    q = gpu_lib.quantize_int8(y.view(2 * m, n))
    p, dy, p8, dy8 = (torch.empty(m, n * w, dtype=torch.bfloat16, device="cuda") for w in (1, 2, 1, 2))

    def step():
        gpu_lib.quantize_int8(y.view(2 * m, n), out=q)
        gpu_lib.gated_fwd(y, out=p), gpu_lib.gated_bwd(y, dp, out=dy)
        gpu_lib.gated_fwd(q, out=p8), gpu_lib.gated_bwd(q, dp, out=dy8)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        new_y, new_dp = (v.cuda() for v in inputs(m, n, torch.bfloat16, 40 + i))
        y.copy_(new_y), dp.copy_(new_dp)
        for v in (p, dy, p8, dy8):
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        q2 = gpu_lib.quantize_int8(new_y.view(2 * m, n))
        assert torch.equal(p, gpu_lib.gated_fwd(new_y)) and torch.equal(dy, gpu_lib.gated_bwd(new_y, new_dp))
        assert torch.equal(p8, gpu_lib.gated_fwd(q2)) and torch.equal(dy8, gpu_lib.gated_bwd(q2, new_dp))
