"""Ends of the ranges of the gated-block and 8-bit backward calls: neighbours that are not finite, sizes past 32-bit
offsets, the longest contractions of each kernel, many row groups a workgroup."""
import numpy as np
import pytest
import torch

import gated_cases as C
import test_gpu_linear_gated as L
import test_gpu_linear_x8 as X
from oracle import gated as OG

pytestmark = pytest.mark.gpu
T = torch.bfloat16


def test_a_block_that_is_not_finite_stays_where_it_is(gpu_lib):
    # 1040 weight rows: the last unit of the transposed contraction holds the start of the next input column
    m, n, k = 300, 1040, 1088
    _, x, dy, h, a, b, alpha = X.layer(gpu_lib, m, n, k, 1, 16, T, 3)
    nbytes = gpu_lib.x8_workspace_bytes(m, n, k, 1, 16)
    assert nbytes > 2 * n * k  # these sizes restore the weight once
    for bad in (float("nan"), float("inf")):
        q = gpu_lib.quantize(C.normal((n, k), 1.5 / k ** 0.5, 3).float().cuda(), double_quant=False)
        q.absmax.view(n, k // 64)[3, 5] = bad  # row 3, input columns 320 .. 383
        clean = gpu_lib.quantize(C.normal((n, k), 1.5 / k ** 0.5, 3).float().cuda(), double_quant=False)
        got, want = (gpu_lib.linear_bwd(v, x, dy, a, b, alpha, h=h)[0] for v in (q, clean))
        rest = torch.ones(k, dtype=torch.bool, device="cuda")
        rest[320:384] = False
        assert not torch.isfinite(got[:, 320:384]).any()
        assert torch.equal(got[:, rest], want[:, rest])


@pytest.mark.parametrize("m", [1, 12, 300])
def test_a_weight_row_that_is_not_finite_stays_where_it_is(gpu_lib, m):
    half, k = 512, 320
    w = C.normal((2 * half, k), 1.5 / k ** 0.5, 3).float().cuda()
    x = C.normal((m, k), 1.0, 4).to(T).cuda()
    q, clean = (gpu_lib.quantize(w, double_quant=False) for _ in range(2))
    q.absmax.view(2 * half, k // 64)[half + 7, 0] = float("nan")  # up's row 7, the first block behind row 6's end
    got, want = gpu_lib.linear_fwd_gated(q, x), gpu_lib.linear_fwd_gated(clean, x)
    assert torch.isnan(got[0][:, 7]).all() and torch.isnan(got[1][:, half + 7]).all()
    for p, v, col in ((got[0], want[0], 7), (got[1], want[1], half + 7)):
        rest = torch.ones(p.shape[1], dtype=torch.bool, device="cuda")
        rest[col] = False
        assert torch.equal(p[:, rest], v[:, rest])


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_gradients_whose_factors_overflow_together(gpu_lib, kind):
    # dP U alone leaves float32, act' is 0 (g = -200) or tiny (g = -80, SiLU: -79 e^-80 = -1.4e-33)
    t = C.TYPES[kind]
    y = torch.tensor([[-200.0, -80.0, 0.0, 1e25, 1e25, 1e25]], dtype=t).cuda()
    dp = torch.tensor([[1e25, 1e25, 1e10]], dtype=t).cuda()
    dg = C.f64(gpu_lib.gated_bwd(y, dp))[0, :3]
    g, u, d = C.f64(y)[0, :3], C.f64(y)[0, 3:], C.f64(dp)[0]
    want = OG.bwd(g, u, d, OG.SILU)[0]
    assert dg[0] == 0
    # sigma's relative error, 2^-21 (1 + 80) in 16 bits and expf's few 2^-24 in 32, and its products' roundings
    rel = 2 * C.half_step(t) + (2.0 ** -14 if kind == "bf16" else 2.0 ** -20)
    assert (np.abs(dg[1:] - want[1:]) <= rel * np.abs(want[1:])).all(), (dg, want)


@pytest.mark.parametrize("how", [dict(double_quant=False), dict(codebook=1), dict(double_quant=2)])
@pytest.mark.parametrize("m", [9, 70])
def test_weight_formats_backward(gpu_lib, m, how):
    n, k = 144, 192
    w, x, dy, h, a, b, alpha = X.layer(gpu_lib, m, n, k, 1, 16, T, 77)
    w = gpu_lib.quantize(C.normal((n, k), 1.5 / k ** 0.5, 77).float().cuda(), **how)
    args = (w, x, dy, h, a, b, alpha)
    for name, v, (want, off) in zip(("dX", "dA", "dB"), X.call(gpu_lib, *args, 1), X.expected(gpu_lib, *args, 1, T)):
        C.check(v, want, off, name)


# the longest contraction that is multiplied from a restored weight, and the first past it
@pytest.mark.parametrize("k", [65536, 65600])
@pytest.mark.parametrize("m", [1, 9, 40])
def test_long_inputs(gpu_lib, m, k):
    w, x, a, b, alpha = L.layer(gpu_lib, m, 256, k, 16, T, 5)
    L.compare(gpu_lib, w, x, a, b, alpha, OG.SILU, T)


@pytest.mark.parametrize("n", [65536, 65552])
def test_long_outputs_backward(gpu_lib, n):
    X.compare(gpu_lib, 40, n, 64, 1, 16, "bf16", 6)


# 16 weight rows a group: 11 groups a workgroup on 256 CUs, in batches of six
@pytest.mark.parametrize("k", [64, 4160])
@pytest.mark.parametrize("m", [1, 16])
def test_many_outputs_of_few_tokens(gpu_lib, m, k):
    half, r = 22528, 8
    gen = torch.Generator(device="cuda").manual_seed(k)
    draw = lambda *shape: torch.empty(shape, device="cuda").normal_(generator=gen)  # noqa: E731
    w = gpu_lib.quantize(draw(2 * half, k) / k ** 0.5)
    x, a, b = draw(m, k).to(T), draw(2 * r, k).to(T) / r, (0.05 * draw(2 * half, r)).to(T)
    p, y, h = gpu_lib.linear_fwd_gated(w, x, a, b, 2.0 * r)
    pick = torch.cat([torch.arange(i, half, 997) for i in (0, 1, 8)] + [torch.arange(half - 40, half)]).unique()
    rows = torch.cat([pick, half + pick]).cuda()
    w64 = gpu_lib.dequantize(w, T)[rows].cpu().double()
    x64, a64, b64 = x.cpu().double(), a.cpu().double(), b[rows].cpu().double()
    v, off = x64 @ w64.t().contiguous(), (x64.abs() @ w64.abs().t().contiguous()) * (k * C.F32)
    h64, h_off = x64 @ a64.t().contiguous(), (x64.abs() @ a64.abs().t().contiguous()) * (k * C.F32)
    for l in range(2):
        cols, slots = slice(l * len(pick), (l + 1) * len(pick)), slice(l * r, (l + 1) * r)
        bt = b64[cols].t().contiguous()
        v[:, cols] += 2 * h64[:, slots] @ bt
        off[:, cols] += (2 * h64[:, slots].abs() * (C.half_step(T) + (r + 2) * C.F32) + 2 * h_off[:, slots]) @ bt.abs()
    v, off = v.numpy(), off.numpy() * 1.01
    C.check(y[:, rows], v, np.abs(v) * C.half_step(T) * (1 + 2 ** -7) + off * 1.01, "Y")
    g, u = v[:, :len(pick)], v[:, len(pick):]
    C.check(p[:, pick.cuda()], OG.fwd(g, u, OG.SILU), C.fwd_bound(g, u, OG.SILU, T, off[:, :len(pick)], off[:, len(pick):]), "P")


# enough weights that 17 to 32 tokens are two decode launches
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("m,r", [(17, 16), (29, 5), (32, 0)])
def test_tokens_by_sixteen(gpu_lib, m, r, kind):
    half, k, t = 5632, 2048, C.TYPES[kind]
    assert gpu_lib.gated_workspace_bytes(m, 2 * half, k, r) < 2 * half * k
    w, x, a, b, alpha = L.layer(gpu_lib, m, half, k, r, t, m)
    L.compare(gpu_lib, w, x, a, b, alpha, OG.SILU, t)
    p, y, h = gpu_lib.linear_fwd_gated(w, x, a, b, alpha)
    q = gpu_lib.linear_fwd_gated(w, x[16:].contiguous(), a, b, alpha)
    assert torch.equal(p[16:], q[0]) and torch.equal(y[16:], q[1]) and (r == 0 or torch.equal(h[16:], q[2]))


def test_products_past_32_bit_offsets(gpu_lib):
    # 9.8e9 products, in launches of 2^30 runs of eight
    m, n = 600_000, 16384
    gen = torch.Generator(device="cuda").manual_seed(1)
    y = torch.empty((m, 2 * n), dtype=T, device="cuda")
    for part in y.split(50_000):
        part.normal_(generator=gen)
    pick = [0, 65_535, 65_536, 131_071, 131_072, 524_287, 524_288, m - 1]
    few = y[pick].clone()
    print(f"forward {m} x {n}", flush=True)
    p = gpu_lib.gated_fwd(y)
    assert torch.equal(p[pick], gpu_lib.gated_fwd(few))
    print("backward in place", flush=True)
    want = gpu_lib.gated_bwd(few, p[pick].contiguous())
    assert torch.equal(gpu_lib.gated_bwd(y, p, out=y)[pick], want)
    del y, p
    m = 140_000
    print(f"8-bit rows {m} x {n}", flush=True)
    codes = torch.randint(-127, 128, (2 * m, n), dtype=torch.int8, device="cuda", generator=gen)
    q = gpu_lib.PackedInt8(2 * m, n, codes, torch.rand(2 * m, device="cuda", generator=gen) / 64)
    pick = [0, 65_535, 65_536, m - 1]
    rows = [r for t in pick for r in (2 * t, 2 * t + 1)]
    few = gpu_lib.PackedInt8(len(rows), n, q.codes[rows].contiguous(), q.scale[rows].contiguous())
    p = gpu_lib.gated_fwd(q)
    assert torch.equal(p[pick], gpu_lib.gated_fwd(few))
    want = gpu_lib.gated_bwd(few, p[pick].contiguous())
    assert torch.equal(gpu_lib.gated_bwd(q, p)[pick], want)


def test_blocks_past_32_bit_offsets(gpu_lib):
    gen = torch.Generator(device="cuda").manual_seed(2)
    m, n, k = 140_000, 16384, 64
    print(f"8-bit block {m} x {n}", flush=True)
    ints = lambda rows: torch.randint(-127, 128, (rows, k), dtype=torch.int8, device="cuda", generator=gen)  # noqa: E731
    w = gpu_lib.PackedInt8(2 * n, k, ints(2 * n), torch.rand(2 * n, device="cuda", generator=gen) / 256)
    x = gpu_lib.PackedInt8(m, k, ints(m), torch.rand(m, device="cuda", generator=gen) / 256)
    pick = [0, 65_535, 65_536, 131_071, 131_072, m - 1]
    p = gpu_lib.int8_linear_fwd_gated(w, x)
    few = gpu_lib.PackedInt8(len(pick), k, x.codes[pick].contiguous(), x.scale[pick].contiguous())
    assert torch.equal(p[pick], gpu_lib.int8_linear_fwd_gated(w, few))
    del p
    m, half, r = 70_000, 16384, 16
    print(f"block {m} x {half}", flush=True)
    w, _, a, b, alpha = L.layer(gpu_lib, 1, half, k, r, T, 9)
    x = torch.empty((m, k), dtype=T, device="cuda").normal_(generator=gen)
    p, y, h = gpu_lib.linear_fwd_gated(w, x, a, b, alpha)
    pick = [0, 32_767, 32_768, 65_535, 65_536, m - 1]
    g, u, h64, dg, du, dh = L.expected(gpu_lib, w, x[pick], a, b, alpha, T)
    C.check(p[pick], OG.fwd(g, u, OG.SILU), C.fwd_bound(g, u, OG.SILU, T, dg, du), "P")
    v, off = np.concatenate([g, u], 1), np.concatenate([dg, du], 1)
    C.check(y[pick], v, np.abs(v) * C.half_step(T) * (1 + 2 ** -7) + off * 1.01, "Y")
    C.check(h[pick], h64, dh + np.abs(h64) * C.F32, "H")


def test_backward_past_32_bit_offsets(gpu_lib):
    gen = torch.Generator(device="cuda").manual_seed(3)
    m, n, k, r = 70_000, 512, 32768, 16
    print(f"backward {m} x {n} x {k}", flush=True)
    w, _, _, _, a, b, alpha = X.layer(gpu_lib, 1, n, k, 2, r, T, 10)
    x = gpu_lib.PackedInt8(m, k, torch.randint(-127, 128, (m, k), dtype=torch.int8, device="cuda", generator=gen),
                           torch.rand(m, device="cuda", generator=gen) / 64)
    dy = torch.empty((m, n), dtype=T, device="cuda").normal_(generator=gen)
    h = torch.empty((m, 2 * r), device="cuda").normal_(generator=gen)
    dx, da, db = X.call(gpu_lib, w, x, dy, h, a, b, alpha, 2)
    pick = [0, 32_767, 32_768, 65_535, 65_536, m - 1]
    few = gpu_lib.PackedInt8(len(pick), k, x.codes[pick].contiguous(), x.scale[pick].contiguous())
    want, off = X.expected(gpu_lib, w, few, dy[pick], h[pick], a, b, alpha, 2, T)[0]
    C.check(dx[pick], want, off, "dX")
    # 128 columns of dA, the last ones among them, over all rows
    cols = [*range(64), *range(k - 64, k)]
    x64 = x.codes[:, cols].cpu().double() * x.scale.cpu().double()[:, None]
    d, b64 = dy.cpu().double(), b.cpu().double()
    for l in range(2):
        rows = slice(l * n // 2, (l + 1) * n // 2)
        dh = 2 * (d[:, rows] @ b64[rows])
        each = 2 * (d[:, rows].abs() @ b64[rows].abs()) * (n * C.F32) + 4 * C.F32 * dh.abs()
        bound = each.t() @ x64.abs() + (dh.abs().t() @ x64.abs()) * ((3 * m + 8) * C.F32)
        C.check(da[l * r:(l + 1) * r][:, cols], (dh.t() @ x64).numpy(), bound.numpy(), "dA")
        h64 = h[:, l * r:(l + 1) * r].cpu().double()
        bound = 2 * (d[:, rows].abs().t() @ h64.abs()) * ((6 * m + 8) * C.F32)
        C.check(db[rows], (2 * d[:, rows].t() @ h64).numpy(), bound.numpy(), "dB")
