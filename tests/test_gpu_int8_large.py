"""Tensors of more than 2^31 elements through the 8-bit and gradient calls:
offsets pass 32 bits. Inputs are drawn on the GPU; sampled rows, the last ones
among them, are compared with the oracle."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import clip as OC
from oracle import int8 as OI

pytestmark = pytest.mark.gpu


def _f32(t):
    return t.detach().float().cpu().numpy()


def _bf16(v):
    import torch

    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16).float().numpy()


@pytest.mark.parametrize("rows,cols", [(70_000, 32_000), (4_400_000, 500)])
def test_rows_past_2_31_elements(gpu_lib, rows, cols):
    import torch

    say(f"[int8 large] rows {rows}x{cols}")
    assert rows * cols > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    gain = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)
    pick = [0, 1, rows // 2, rows - 2, rows - 1]
    host = _f32(x[pick])
    q = gpu_lib.quantize_int8(x)
    v = gpu_lib.dequantize_int8(q)
    torch.cuda.synchronize()
    codes, scale = OI.quantize(host)
    assert np.array_equal(q.codes[pick].cpu().numpy()[:, :cols], codes)
    assert np.array_equal(q.scale[pick].cpu().numpy(), scale)
    assert np.array_equal(_f32(v[pick]), _bf16(OI.dequantize(codes, scale)))
    del v
    say("   norm in place")
    gpu_lib.rmsnorm_int8(x, gain, 1e-5, residual=x, residual_out=x, out=q)
    torch.cuda.synchronize()
    codes, scale, h = OI.rmsnorm(host, _f32(gain), 1e-5, host)
    assert np.array_equal(q.codes[pick].cpu().numpy()[:, :cols], codes)
    got = q.scale[pick].cpu().numpy()
    assert np.all(np.abs(got.astype(np.float64) - scale) <= 2.0 ** -23 * scale)
    assert np.array_equal(_f32(x[pick]), _bf16(h))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_longest_rows(gpu_lib, dtype):
    import torch

    rows, cols = 3, 1 << 22
    say(f"[int8 large] {rows} rows of {cols} {dtype}")
    x = torch.from_numpy(np.random.default_rng(3).standard_normal((rows, cols)).astype(np.float32))
    x = x.to(getattr(torch, dtype))
    codes, scale = OI.quantize(x.float().numpy())
    q = gpu_lib.quantize_int8(x.cuda())
    n, _ = gpu_lib.rmsnorm_int8(x.cuda(), torch.ones(cols, device="cuda"), 1e-5)
    torch.cuda.synchronize()
    assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.scale.cpu().numpy(), scale)
    codes, scale, _ = OI.rmsnorm(x.float().numpy(), np.ones(cols, np.float32), 1e-5)
    got = n.scale.cpu().numpy()
    assert np.array_equal(n.codes.cpu().numpy(), codes)
    assert np.all(np.abs(got.astype(np.float64) - scale) <= 2.0 ** -23 * scale)
    with pytest.raises(ValueError, match="longer than"):
        gpu_lib.quantize_int8(torch.empty((1, cols + 1), device="cuda"))


@pytest.mark.parametrize("m,n,k", [(40_000, 60_000, 64), (16, 1_000_000, 4096), (600_000, 64, 4096)])
def test_product_past_2_31(gpu_lib, m, n, k):
    """More than 2^31 outputs, weight codes and token codes."""
    import torch

    say(f"[int8 large] product {m}x{n}x{k}")
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randint(-127, 128, (n, k), dtype=torch.int8, device="cuda", generator=g)
    x = torch.randint(-127, 128, (m, k), dtype=torch.int8, device="cuda", generator=g)
    sw, sx = torch.rand(n, device="cuda", generator=g) + 0.5, torch.rand(m, device="cuda", generator=g) + 0.5
    y = gpu_lib.int8_linear_fwd(gpu_lib.PackedInt8(n, k, w, sw), gpu_lib.PackedInt8(m, k, x, sx))
    torch.cuda.synchronize()
    rows = sorted({0, m // 2, m - 1})
    step = max(1, n // 5000)
    cols = torch.cat([torch.arange(0, n, step), torch.arange(max(0, n - 300), n)]).cuda()
    want = OI.linear(w[cols].cpu().numpy(), sw[cols].cpu().numpy(), x[rows].cpu().numpy(), sx[rows].cpu().numpy())
    assert np.array_equal(_f32(y[rows][:, cols]), _bf16(want))


def test_gradient_past_2_31_elements(gpu_lib):
    """One long gradient between two short ones: its last elements and the short
    one behind it are scaled, and the norm counts them. The squares of the long
    one are equal, so the norm is known."""
    import torch

    n = 2 ** 31 + 5001
    say(f"[grad clip large] {n} elements")
    a = torch.full((1000,), 3.0, dtype=torch.bfloat16, device="cuda")
    b = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    c = torch.full((777,), 5.0, dtype=torch.bfloat16, device="cuda")
    total = (9.0 * 1000 + n * 2.0 ** -20 + 25.0 * 777) ** 0.5
    out = torch.empty(1000 + n + 777, dtype=torch.bfloat16, device="cuda")
    norm = gpu_lib.grad_clip([a, b, c], 1.0, out=out)
    f = OC.factor(total, 1.0)
    torch.cuda.synchronize()
    # the sum in 64 bits: relative error below 2^31 2^-53
    assert abs(float(norm) - total) <= 2.0 ** -21 * total
    # one step of the factor's rounding may move an element's by one of its own
    near = lambda t, v: bool((t.float() - float(v)).abs().max() <= 2.0 ** -8 * float(v))  # noqa: E731
    assert near(out[:1000], 3 * f) and near(out[1000 + n:], 5 * f)
    for s in (slice(1000, 6000), slice(2 ** 31 - 100, 2 ** 31 + 100), slice(1000 + n - 5000, 1000 + n)):
        assert near(out[s], 2.0 ** -10 * f)
    assert torch.equal(out[1000:1000 + n].min(), out[1000:1000 + n].max())
