"""The backward calls from an input kept as 8-bit rows, against float64."""
import numpy as np
import pytest
import torch

import gated_cases as C

pytestmark = pytest.mark.gpu


def layer(lib, m, n, k, parts, r, t, seed):
    w = lib.quantize(C.normal((n, k), 1.5 / k ** 0.5, seed).float().cuda())
    x = lib.quantize_int8(C.normal((m, k), 1.0, seed + 1).to(t).cuda())
    dy = C.normal((m, n), 1.0, seed + 2).to(t).cuda()
    h = C.normal((m, parts * r), 2.0, seed + 3).float().cuda()
    a = C.normal((parts * r, k), 1.0 / max(r, 1), seed + 4).to(t).cuda()
    b = C.normal((n, r), 0.05, seed + 5).to(t).cuda()
    return w, x, dy, h, a, b, 2.0 * r


def expected(lib, w, x, dy, h, a, b, alpha, parts, t):
    """(value, bound) of dX, dA and dB."""
    m, n, k, r = x.n, w.n, w.k, b.shape[1]
    s = alpha / r
    w64 = lib.dequantize(w, t).cpu().double()
    d, a64, b64, h64 = dy.cpu().double(), a.cpu().double(), b.cpu().double(), h.cpu().double()
    x64 = x.codes[:, :k].cpu().double() * x.scale.cpu().double()[:, None]
    dx, dx_off = d @ w64, d.abs() @ w64.abs() * (n * C.F32)
    da, da_off, db, db_off = [], [], [], []
    for l in range(parts):
        rows, slots = slice(l * (n // parts), (l + 1) * (n // parts)), slice(l * r, (l + 1) * r)
        dl = d[:, rows].contiguous()
        dh = s * (dl @ b64[rows])
        # float32 sums over n (grouped: over the zeros of the other parts too), scaled
        dh_off = s * (dl.abs() @ b64[rows].abs()) * (n * C.F32) + 2 * C.F32 * dh.abs()
        dx += dh @ a64[slots]
        low = dh.abs() * C.half_step(t) + dh_off + C.tiny(t)  # dH in 16 bits in dX
        dx_off += low @ a64[slots].abs() + (dh.abs() @ a64[slots].abs()) * (r * C.F32)
        da.append(dh.t().contiguous() @ x64)
        # dH x scale is one more rounding, the sum over m tokens of three exact products each
        each = dh_off + dh.abs() * (2 * C.F32)
        da_off.append(each.t().contiguous() @ x64.abs() + (dh.abs().t().contiguous() @ x64.abs()) * ((3 * m + 8) * C.F32))
        db.append(s * (dl.t().contiguous() @ h64[:, slots]))
        db_off.append(s * (dl.abs().t().contiguous() @ h64[:, slots].abs()) * ((6 * m + 8) * C.F32))
    dx, dx_off = dx.numpy(), dx_off.numpy() * 1.01
    return ((dx, np.abs(dx) * C.half_step(t) * (1 + 2 ** -7) + dx_off + C.tiny(t)),
            (torch.cat(da).numpy(), torch.cat(da_off).numpy() + 1e-30), (torch.cat(db).numpy(), torch.cat(db_off).numpy() + 1e-30))


def call(lib, w, x, dy, h, a, b, alpha, parts, **more):
    if parts == 1:
        return lib.linear_bwd(w, x, dy, a, b, alpha, h=h, **more)
    return lib.linear_bwd_grouped(w, [w.n // parts] * parts, x, dy, a, b, alpha, h=h, **more)


def compare(lib, m, n, k, parts, r, kind, seed):
    t = C.TYPES[kind]
    args = layer(lib, m, n, k, parts, r, t, seed)
    got = call(lib, *args, parts)
    for name, v, (want, off) in zip(("dX", "dA", "dB"), got, expected(lib, *args, parts, t)):
        C.check(v, want, off, name)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("r", [1, 5, 16, 24, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 16, 64), (33, 144, 192), (300, 272, 320)])
def test_one_linear(gpu_lib, m, n, k, r, kind):
    compare(gpu_lib, m, n, k, 1, r, kind, m + r)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("parts,r", [(2, 16), (3, 16), (4, 32), (2, 64)])
@pytest.mark.parametrize("m", [5, 257])
def test_grouped(gpu_lib, m, parts, r, kind):
    compare(gpu_lib, m, 256 * parts, 320, parts, r, kind, m + r)


# more rows than one split takes, and columns enough for a single one
@pytest.mark.parametrize("m,n,k,r", [(2048, 256, 512, 16), (1111, 4096, 1088, 8), (600, 1024, 40000 // 64 * 64, 16)])
def test_splits(gpu_lib, m, n, k, r):
    compare(gpu_lib, m, n, k, 1, r, "bf16", m)


def test_rows_longer_than_the_input(gpu_lib):
    w, x, dy, h, a, b, alpha = layer(gpu_lib, 40, 128, 192, 1, 16, torch.bfloat16, 2)
    wide = torch.full((40, 320), 77, dtype=torch.int8, device="cuda")  # codes behind k are not read
    wide[:, :192] = x.codes
    y = gpu_lib.PackedInt8(40, 192, wide, x.scale)
    assert all(torch.equal(p, q) for p, q in zip(call(gpu_lib, w, x, dy, h, a, b, alpha, 1), call(gpu_lib, w, y, dy, h, a, b, alpha, 1)))


def test_repeats_and_outputs(gpu_lib):
    args = layer(gpu_lib, 700, 256, 448, 1, 16, torch.bfloat16, 3)
    dx, da, db = call(gpu_lib, *args, 1)
    rooms = [torch.full((v.numel() + 256,), 5.0, dtype=v.dtype, device="cuda") for v in (dx, da, db)]
    outs = [q[: v.numel()].view(v.shape) for q, v in zip(rooms, (dx, da, db))]
    nbytes = gpu_lib.x8_workspace_bytes(700, 256, 448, 1, 16)
    ws = torch.full((nbytes + 256,), 9, dtype=torch.uint8, device="cuda")
    got = call(gpu_lib, *args, 1, dx=outs[0], da=outs[1], db=outs[2], ws=ws[:nbytes])
    assert all(torch.equal(p, q) for p, q in zip(got, (dx, da, db)))
    assert all((q[-256:] == 5.0).all() for q in rooms) and (ws[nbytes:] == 9).all()
    none, da2, db2 = call(gpu_lib, *args, 1, need_dx=False)
    assert none is None and torch.equal(da2, da) and torch.equal(db2, db)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k,r", [(17, 272, 576, 16), (300, 1040, 1088, 5)])
def test_workspace_without_the_restored_weight(gpu_lib, m, n, k, r, kind):
    # the call restores the weight as it multiplies; both ways are within the bounds
    t = C.TYPES[kind]
    args = layer(gpu_lib, m, n, k, 1, r, t, 12)
    nbytes = gpu_lib.x8_workspace_bytes(m, n, k, 1, r)
    without = nbytes - 2 * n * k
    ws = torch.full((without + 256,), 9, dtype=torch.uint8, device="cuda")
    want = expected(gpu_lib, *args, 1, t)
    for room in (ws[:without], torch.empty(nbytes, dtype=torch.uint8, device="cuda")):
        for name, v, (value, off) in zip(("dX", "dA", "dB"), call(gpu_lib, *args, 1, ws=room), want):
            C.check(v, value, off, name)
    assert (ws[without:] == 9).all()
    with pytest.raises(gpu_lib.QloraError, match="WORKSPACE"):
        call(gpu_lib, *args, 1, ws=ws[:without - 1])


@pytest.mark.parametrize("m,n,k,r", [(2050, 208, 1088, 16), (1030, 80, 2816, 0), (700, 4112, 192, 5), (40, 8208, 320, 24)])
def test_tiles_of_the_restored_weight(gpu_lib, m, n, k, r):
    if r:
        compare(gpu_lib, m, n, k, 1, r, "fp16", m)
    else:
        w, x, dy, _, _, _, _ = layer(gpu_lib, m, n, k, 1, 1, torch.bfloat16, m)
        d, w64 = dy.cpu().double(), gpu_lib.dequantize(w, torch.bfloat16).cpu().double()
        dx = (d @ w64).numpy()
        bound = np.abs(dx) * C.half_step(torch.bfloat16) * (1 + 2 ** -7) + (d.abs() @ w64.abs()).numpy() * (n * C.F32) * 1.01
        C.check(gpu_lib.linear_bwd(w, x, dy)[0], dx, bound, "dX")


def test_agrees_with_the_16_bit_input(gpu_lib):
    # codes of whole numbers over a scale of one are exact in bf16: the same X to both calls
    w, x, dy, h, a, b, alpha = layer(gpu_lib, 128, 256, 320, 1, 16, torch.bfloat16, 5)
    x.scale.fill_(1.0)
    x16 = x.codes[:, :320].to(torch.bfloat16)
    got, want = call(gpu_lib, w, x, dy, h, a, b, alpha, 1), gpu_lib.linear_bwd(w, x16, dy, a, b, alpha, h=h)
    # dX: both calls are within the same bound of the float64 value (half a step of bf16 and the float32 sums'
    # roundings, whose order may differ), so within twice that of each other
    value, bound = expected(gpu_lib, w, x, dy, h, a, b, alpha, 1, torch.bfloat16)[0]
    C.check(got[0], C.f64(want[0]), 2 * bound, "dX")
    for p, q in zip(got[1:], want[1:]):
        assert (p - q).abs().max() <= 1e-4 * q.abs().max()  # the 16-bit call's own bound


def test_rows_that_are_not_finite(gpu_lib):
    w, x, dy, h, a, b, alpha = layer(gpu_lib, 40, 128, 192, 1, 16, torch.bfloat16, 8)
    x.scale[3] = float("nan")
    dx, da, db = call(gpu_lib, w, x, dy, h, a, b, alpha, 1)
    assert torch.isnan(da).all() and torch.isfinite(dx).all() and torch.isfinite(db).all()


def test_no_tokens_and_no_adapter(gpu_lib):
    w, x, dy, h, a, b, alpha = layer(gpu_lib, 8, 128, 192, 1, 16, torch.bfloat16, 9)
    none = gpu_lib.PackedInt8(0, 192, x.codes[:0], x.scale[:0])
    dx, da, db = call(gpu_lib, w, none, dy[:0], h[:0], a, b, alpha, 1)
    assert dx.shape == (0, 192) and not da.any() and not db.any()
    dx, da, db = gpu_lib.linear_bwd(w, x, dy)
    want = gpu_lib.linear_bwd(w, torch.zeros(8, 192, dtype=torch.bfloat16, device="cuda"), dy)[0]
    assert da is None and db is None and torch.equal(dx, want)


def test_captured_with_eager_calls_between(gpu_lib):
    t = torch.bfloat16
    w, x, dy, h, a, b, alpha = layer(gpu_lib, 300, 512, 320, 2, 16, t, 10)
    dx, da, db = torch.empty(300, 320, dtype=t, device="cuda"), torch.empty(32, 320, device="cuda"), torch.empty(512, 16, device="cuda")
    ws = torch.empty(gpu_lib.x8_workspace_bytes(300, 512, 320, 2, 16), dtype=torch.uint8, device="cuda")
    step = lambda: call(gpu_lib, w, x, dy, h, a, b, alpha, 2, dx=dx, da=da, db=db, ws=ws)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        dy.copy_(C.normal((300, 512), 1.0, 50 + i).to(t).cuda())
        for v in (dx, da, db):
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = call(gpu_lib, w, x, dy, h, a, b, alpha, 2)
        assert all(torch.equal(p, q) for p, q in zip((dx, da, db), want))
