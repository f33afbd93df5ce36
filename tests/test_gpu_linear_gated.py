"""The gated block over an NF4 weight with adapters, against float64 over the restored weight."""
import numpy as np
import pytest
import torch

import gated_cases as C
from oracle import gated as OG

pytestmark = pytest.mark.gpu


def layer(lib, m, half, k, r, t, seed, **how):
    """(packed weight, x, a, b, alpha) on the GPU."""
    w = lib.quantize(C.normal((2 * half, k), 1.5 / k ** 0.5, seed).float().cuda(), **how)
    x = C.normal((m, k), 1.0, seed + 1).to(t).cuda()
    a = (C.normal((2 * r, k), 1.0 / r, seed + 2).to(t).cuda()) if r else None
    b = (C.normal((2 * half, r), 0.05, seed + 3).to(t).cuda()) if r else None
    return w, x, a, b, 2.0 * r


def expected(lib, w, x, a, b, alpha, t):
    """(gate, up, H) in float64 and how far float32 sums and a 16-bit s H leave them."""
    half = w.n // 2
    x64, w64 = x.cpu().double(), lib.dequantize(w, t).cpu().double()
    y, mag = x64 @ w64.t().contiguous(), x64.abs() @ w64.abs().t().contiguous()
    off = mag * (w.k * C.F32)
    if a is None:
        y, off = y.numpy(), off.numpy()
        return y[:, :half], y[:, half:], None, off[:, :half], off[:, half:], None
    r = b.shape[1]
    s = alpha / r
    a64, b64 = a.cpu().double(), b.cpu().double()
    h, hoff = x64 @ a64.t().contiguous(), (x64.abs() @ a64.abs().t().contiguous()) * (w.k * C.F32)
    for l in range(2):
        rows, slots = slice(l * half, (l + 1) * half), slice(l * r, (l + 1) * r)
        bt = b64[rows].t().contiguous()
        y[:, rows] += s * h[:, slots] @ bt
        # s H enters the matrix cores in 16 bits (fp16: its subnormals too); r more terms
        low = (s * h[:, slots]).abs() * (C.half_step(t) + (r + 2) * C.F32) + s * hoff[:, slots] + C.tiny(t)
        off[:, rows] += low @ bt.abs()
    y, off = y.numpy(), off.numpy() * 1.01
    return y[:, :half], y[:, half:], h.numpy(), off[:, :half], off[:, half:], hoff.numpy()


def compare(lib, w, x, a, b, alpha, act, t, keep=True):
    p, y, h = lib.linear_fwd_gated(w, x, a, b, alpha, act, want_y=keep, want_h=keep)
    g, u, h64, dg, du, dh = expected(lib, w, x, a, b, alpha, t)
    C.check(p, OG.fwd(g, u, act), C.fwd_bound(g, u, act, t, dg, du), "P")
    if not keep:
        assert y is None and h is None
        return
    v, off = np.concatenate([g, u], 1), np.concatenate([dg, du], 1)
    C.check(y, v, np.abs(v) * C.half_step(t) * (1 + 2 ** -7) + off * 1.01 + C.tiny(t), "Y")
    if a is None:
        assert h is None
    else:
        C.check(h, h64, dh + np.abs(h64) * C.F32, "H")


MS = [1, 2, 3, 16, 17, 40, 256, 300]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("r", [0, 5, 8, 16, 64])
@pytest.mark.parametrize("m", MS)
def test_block(gpu_lib, m, r, kind):
    t = C.TYPES[kind]
    w, x, a, b, alpha = layer(gpu_lib, m, 512, 320, r, t, m + r)
    compare(gpu_lib, w, x, a, b, alpha, r % 2, t)


@pytest.mark.parametrize("half,k", [(256, 64), (768, 4096), (256, 4160), (1280, 1088), (256, 12352)])
@pytest.mark.parametrize("m", [1, 7, 70])
def test_sizes(gpu_lib, m, half, k):
    w, x, a, b, alpha = layer(gpu_lib, m, half, k, 16, torch.bfloat16, half + k)
    compare(gpu_lib, w, x, a, b, alpha, OG.GELU, torch.bfloat16)


@pytest.mark.parametrize("how", [dict(double_quant=False), dict(codebook=1), dict(double_quant=2)])
@pytest.mark.parametrize("m", [1, 5, 33])
def test_weight_formats(gpu_lib, m, how):
    w, x, a, b, alpha = layer(gpu_lib, m, 256, 192, 8, torch.bfloat16, 77, **how)
    if how.get("double_quant") == 2:
        assert w.double_quant == 2
    compare(gpu_lib, w, x, a, b, alpha, OG.SILU, torch.bfloat16)


@pytest.mark.parametrize("m", [1, 2, 9, 65])
def test_product_alone_is_the_same(gpu_lib, m):
    w, x, a, b, alpha = layer(gpu_lib, m, 512, 256, 16, torch.bfloat16, 4)
    compare(gpu_lib, w, x, a, b, alpha, OG.SILU, torch.bfloat16, keep=False)
    p, y, h = gpu_lib.linear_fwd_gated(w, x, a, b, alpha)
    q, none, none2 = gpu_lib.linear_fwd_gated(w, x, a, b, alpha, want_y=False, want_h=False)
    assert none is None and none2 is None and torch.equal(p, q)
    p2, y2, h2 = gpu_lib.linear_fwd_gated(w, x, a, b, alpha)
    assert torch.equal(p, p2) and torch.equal(y, y2) and torch.equal(h, h2)


def test_model_sizes(gpu_lib):
    for m, half, k, r in ((1, 11008, 4096, 16), (13, 11008, 4096, 16), (40, 11008, 4096, 16)):
        w, x, a, b, alpha = layer(gpu_lib, m, half, k, r, torch.bfloat16, 6)
        compare(gpu_lib, w, x, a, b, alpha, OG.SILU, torch.bfloat16)


@pytest.mark.parametrize("m", [1, 4, 50])
def test_outputs_end_where_they_end(gpu_lib, m):
    t = torch.bfloat16
    w, x, a, b, alpha = layer(gpu_lib, m, 256, 128, 16, t, 9)
    rooms = [torch.full((m * c + 256,), 5.0, dtype=d, device="cuda") for c, d in ((256, t), (512, t), (32, torch.float32))]
    p, y, h = (v[: m * c].view(m, c) for v, c in zip(rooms, (256, 512, 32)))
    nbytes = gpu_lib.gated_workspace_bytes(m, 512, 128, 16)
    ws = torch.full((nbytes + 256,), 9, dtype=torch.uint8, device="cuda")
    got = gpu_lib.linear_fwd_gated(w, x, a, b, alpha, out=p, y_out=y, h_out=h, ws=ws[:nbytes] if nbytes else None)
    assert got[0] is p and got[1] is y and got[2] is h
    want = gpu_lib.linear_fwd_gated(w, x, a, b, alpha)
    assert all(torch.equal(v, q) for v, q in zip(got, want))
    assert all((v[-256:] == 5.0).all() for v in rooms) and (ws[nbytes:] == 9).all()


def test_captured_with_eager_calls_between(gpu_lib):
    t = torch.bfloat16
    for m in (1, 12, 48):
        w, x, a, b, alpha = layer(gpu_lib, m, 512, 256, 16, t, m)
        p, y = torch.empty(m, 512, dtype=t, device="cuda"), torch.empty(m, 1024, dtype=t, device="cuda")
        h = torch.empty(m, 32, device="cuda")
        ws = torch.empty(max(1, gpu_lib.gated_workspace_bytes(m, 1024, 256, 16)), dtype=torch.uint8, device="cuda")
        call = lambda: gpu_lib.linear_fwd_gated(w, x, a, b, alpha, out=p, y_out=y, h_out=h, ws=ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for i in range(3):
            x.copy_(C.normal((m, 256), 1.0, 100 + i).to(t).cuda())
            p.fill_(float("nan")), y.fill_(float("nan")), h.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            want = gpu_lib.linear_fwd_gated(w, x, a, b, alpha)
            assert torch.equal(p, want[0]) and torch.equal(y, want[1]) and torch.equal(h, want[2])


@pytest.mark.parametrize("m", [17, 70, 300])
@pytest.mark.parametrize("r", [0, 8, 16, 64])
def test_workspace_without_the_restored_weight(gpu_lib, m, r):
    # the call restores the weight as it multiplies; both ways are within the bounds
    t, half, k = torch.bfloat16, 512, 320
    w, x, a, b, alpha = layer(gpu_lib, m, half, k, r, t, 31)
    nbytes = gpu_lib.gated_workspace_bytes(m, 2 * half, k, r)
    without = nbytes - 2 * half * k * 2
    assert without >= 0  # these sizes restore it once
    ws = torch.full((without + 256,), 9, dtype=torch.uint8, device="cuda")
    g, u, _, dg, du, _ = expected(gpu_lib, w, x, a, b, alpha, t)
    for size in (without, nbytes):
        room = ws[:without] if size == without else torch.empty(size, dtype=torch.uint8, device="cuda")
        p, y, _ = gpu_lib.linear_fwd_gated(w, x, a, b, alpha, OG.GELU, ws=room if size else None)
        C.check(p, OG.fwd(g, u, OG.GELU), C.fwd_bound(g, u, OG.GELU, t, dg, du), "P")
        v, off = np.concatenate([g, u], 1), np.concatenate([dg, du], 1)
        C.check(y, v, np.abs(v) * C.half_step(t) * (1 + 2 ** -7) + off * 1.01 + C.tiny(t), "Y")
    assert (ws[without:] == 9).all()
    if without:
        with pytest.raises(gpu_lib.QloraError, match="WORKSPACE"):
            gpu_lib.linear_fwd_gated(w, x, a, b, alpha, ws=ws[:without - 1])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("m,half,k,r", [(2100, 1024, 1088, 16), (1030, 2816, 256, 5), (600, 5632, 192, 0), (200, 512, 8192, 24)])
def test_tiles_of_the_restored_weight(gpu_lib, m, half, k, r, kind):
    t = C.TYPES[kind]
    w, x, a, b, alpha = layer(gpu_lib, m, half, k, r, t, m)
    compare(gpu_lib, w, x, a, b, alpha, OG.SILU, t)


def test_no_tokens(gpu_lib):
    w, x, a, b, alpha = layer(gpu_lib, 1, 256, 64, 16, torch.bfloat16, 1)
    p, y, h = gpu_lib.linear_fwd_gated(w, x[:0], a, b, alpha)
    assert p.shape == (0, 256) and y.shape == (0, 512) and h.shape == (0, 32)
