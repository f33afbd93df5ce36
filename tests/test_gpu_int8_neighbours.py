"""Buffers of the 8-bit row calls that touch without overlapping: results are
those on buffers of their own, bit for bit."""
import pytest

from gpu_cases import say

pytestmark = pytest.mark.gpu


def test_rows_in_one_allocation(gpu_lib):
    import torch

    rows, cols, ld = 40, 96, 128
    say("[int8] neighbouring buffers")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    r = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    gain = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    want, h = gpu_lib.rmsnorm_int8(x, gain, residual=r)
    want_q = gpu_lib.quantize_int8(x)
    want_v = gpu_lib.dequantize_int8(want_q)

    pool = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    at = 0

    def take(shape, dtype):
        nonlocal at
        n = torch.Size(shape).numel() * dtype.itemsize
        t = pool[at:at + n].view(dtype).view(shape)
        at += n
        assert at % 16 == 0 and at <= pool.numel()
        return t

    # x | codes | h | scale | residual | gain | values, each behind the last
    px, codes, ph = take((rows, cols), x.dtype), take((rows, ld), torch.int8), take((rows, cols), x.dtype)
    scale, pr, pg = take((rows,), torch.float32), take((rows, cols), x.dtype), take((cols,), x.dtype)
    pv = take((rows, cols), x.dtype)
    px.copy_(x), pr.copy_(r), pg.copy_(gain)
    out = gpu_lib.PackedInt8(rows, cols, codes, scale)
    gpu_lib.rmsnorm_int8(px, pg, residual=pr, residual_out=ph, out=out)
    torch.cuda.synchronize()
    assert torch.equal(codes, want.codes) and torch.equal(scale, want.scale) and torch.equal(ph, h)
    gpu_lib.quantize_int8(px, out=out)
    gpu_lib.dequantize_int8(out, out=pv)
    torch.cuda.synchronize()
    assert torch.equal(codes, want_q.codes) and torch.equal(scale, want_q.scale) and torch.equal(pv, want_v)
    # in place: h over the residual, and over x
    for into in (pr, px):
        keep = into.clone()
        gpu_lib.rmsnorm_int8(px, pg, residual=pr, residual_out=into, out=out)
        torch.cuda.synchronize()
        assert torch.equal(into, h) and torch.equal(codes, want.codes) and torch.equal(scale, want.scale)
        into.copy_(keep)


def test_gradients_norm_and_workspace_in_one_allocation(gpu_lib):
    """gradient | norm | workspace | gradient, an empty tensor's address among
    them; then a workspace larger than needed whose end holds the norm."""
    import torch

    say("[grad clip] neighbouring buffers")
    gen = torch.Generator(device="cuda").manual_seed(2)
    host = [torch.randn(n, generator=gen, device="cuda") for n in (100, 5000)]
    want = torch.empty(5100, device="cuda")
    norm = gpu_lib.grad_clip(host, 0.5, out=want)
    need = gpu_lib.GradList(host).ws_bytes
    assert need % 16 == 0
    pool = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    a = pool[:400].view(torch.float32)
    pn = pool[400:404].view(torch.float32)
    ws = pool[416:416 + need]
    b = pool[416 + need:416 + need + 20000].view(torch.float32)
    inside = ws[8:8].view(torch.float32)
    a.copy_(host[0]), b.copy_(host[1])
    assert gpu_lib.grad_norm([a, inside, b], norm=pn, ws=ws) is pn
    torch.cuda.synchronize()
    assert torch.equal(pn[0], norm)
    pn.zero_()
    gpu_lib.grad_clip([a, inside, b], 0.5, norm=pn, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(pn[0], norm) and torch.equal(torch.cat([a, b]), want)
    long = torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
    tail = long[need:need + 4].view(torch.float32)
    assert torch.equal(gpu_lib.grad_norm(host, norm=tail, ws=long)[0], norm)


def test_views_of_rows(gpu_lib):
    """Some rows of a packed input as they lie, where their scales start at 16
    bytes; elsewhere the call refuses them and takes a copy of the scales."""
    import torch

    m, n, k = 11, 70, 130
    say("[int8] views of rows")
    g = torch.Generator(device="cuda").manual_seed(3)
    w = gpu_lib.quantize_int8(torch.randn(n, k, generator=g, device="cuda"))
    x = gpu_lib.quantize_int8(torch.randn(m, k, generator=g, device="cuda"))
    whole = gpu_lib.int8_linear_fwd(w, x, torch.float32)
    for i in range(m):
        part = gpu_lib.PackedInt8(m - i, k, x.codes[i:], x.scale[i:])
        if i % 4:
            with pytest.raises(gpu_lib.QloraError, match="ALIGN"):
                gpu_lib.int8_linear_fwd(w, part, torch.float32)
            part.scale = part.scale.clone()
        assert torch.equal(gpu_lib.int8_linear_fwd(w, part, torch.float32), whole[i:])
