"""Host checks of the 8-bit and gradient calls (no GPU): the C ABI refuses bad
arguments before any launch, and the binding refuses tensors that do not match
what a call assumes. Fake aligned addresses and CPU tensors stand in: every
case here ends before a kernel."""
import ctypes

import pytest
import torch

from bit_nf4_quantized_18_amd import binding as B

P = 1 << 20
BF16, F32, F16 = B.QLORA_BF16, B.QLORA_F32, B.QLORA_F16


def test_quantize_and_dequantize_argument_errors():
    lib = B.load()
    q = lambda x=P, t=BF16, rows=4, cols=100, codes=P, ld=128, scale=P: lib.qlora_int8_quantize(  # noqa: E731
        x, t, rows, cols, codes, ld, scale, None)
    d = lambda x=P, t=BF16, rows=4, cols=100, codes=P, ld=128, scale=P: lib.qlora_int8_dequantize(  # noqa: E731
        codes, ld, scale, rows, cols, t, x, None)
    for f in (q, d):
        assert f(t=3) == -4 and f(t=-1) == -4
        assert f(x=None) == -1 and f(codes=None) == -1 and f(scale=None) == -1
        assert f(x=P + 2) == -3 and f(codes=P + 8) == -3 and f(scale=P + 4) == -3
        assert f(cols=0) == -2 and f(cols=129) == -2 and f(ld=100) == -2 and f(rows=-1) == -2
        assert f(rows=1 << 31) == -2 and f(cols=100, ld=(1 << 22) + 64) == -2
        assert f(rows=0, x=None, codes=None, scale=None) == 0


def test_rmsnorm_argument_errors():
    lib = B.load()

    def f(x=P, res=P, gain=P, t=BF16, gt=BF16, rows=4, cols=100, eps=1e-6, out=P, codes=P, ld=128, scale=P):
        return lib.qlora_rmsnorm_int8(x, res, gain, t, gt, rows, cols, eps, out, codes, ld, scale, None)

    assert f(t=5) == -4 and f(gt=F16) == -4 and f(t=F32, gt=BF16) == -4
    assert f(eps=-1e-6) == -4 and f(eps=float("nan")) == -4 and f(eps=float("inf")) == -4
    assert f(x=None) == -1 and f(gain=None) == -1 and f(codes=None) == -1 and f(scale=None) == -1
    assert f(out=None) == -1  # a residual without its output
    for name in ("x", "res", "gain", "out", "codes", "scale"):
        assert f(**{name: P + 4}) == -3
    assert f(cols=0) == -2 and f(ld=64) == -2 and f(ld=120) == -2 and f(rows=-2) == -2
    assert f(rows=0, x=None, gain=None) == 0


def test_linear_argument_errors():
    lib = B.load()

    def f(w=P, sw=P, n=64, k=128, x=P, sx=P, m=4, t=BF16, y=P):
        return lib.qlora_int8_linear_fwd(w, sw, n, k, x, sx, m, t, y, None)

    assert f(t=9) == -4
    for name in ("w", "sw", "x", "sx", "y"):
        assert f(**{name: None}) == -1
        assert f(**{name: P + 4}) == -3
    assert f(n=0) == -2 and f(k=0) == -2 and f(k=100) == -2 and f(m=-1) == -2 and f(m=1 << 31) == -2
    assert f(k=131072) == -2 and f(n=(1 << 22) + 1) == -2  # 131072 128^2 = 2^31: the sum could wrap
    assert f(m=0, x=None, sx=None, y=None) == 0
    assert f(n=1 << 22, m=(1 << 31) - 1) == -2  # more tiles than a launch takes


def _grads(sizes, at=None):
    n = len(sizes)
    ptr = (ctypes.c_void_p * max(n, 1))(*(at if at is not None else [P + i * (1 << 24) for i in range(n)]))
    return ptr, (ctypes.c_int64 * max(n, 1))(*sizes), n


def test_grad_argument_errors():
    lib = B.load()
    ptr, num, n = _grads([100, 0, 50])
    need = lib.qlora_grad_workspace_bytes(num, n)
    assert need > 0

    def norm(p=ptr, s=num, c=n, t=F32, out=P, ws=P, nbytes=need):
        return lib.qlora_grad_norm(p, s, c, t, out, ws, nbytes, None)

    def clip(p=ptr, s=num, c=n, t=F32, mx=1.0, o=None, out=P, ws=P, nbytes=need):
        return lib.qlora_grad_clip(p, s, c, t, mx, o, out, ws, nbytes, None)

    for f in (norm, clip):
        assert f(t=3) == -4 and f(p=None) == -1 and f(s=None) == -1 and f(out=None) == -1
        assert f(out=P + 2) == -3 and f(ws=P + 8) == -3
        assert f(nbytes=need - 1) == -5 and f(ws=None) == -5
        assert f(c=-1) == -2 and f(c=(1 << 20) + 1) == -2
        p2, s2, c2 = _grads([100, -1])
        assert f(p=p2, s=s2, c=c2) == -2
        p2, s2, c2 = _grads([1 << 40, 1])
        assert f(p=p2, s=s2, c=c2) == -2
        p2, s2, c2 = _grads([100, 50], [P, 0])
        assert f(p=p2, s=s2, c=c2) == -1
        p2, s2, c2 = _grads([100, 50], [P, P + 4 * 1000 + 2])
        assert f(p=p2, s=s2, c=c2) == -3
    assert clip(mx=-0.5) == -4 and clip(mx=float("nan")) == -4
    # overlaps: the same tensor twice, one element shared, the output over a gradient
    for at in ([P, P], [P, P + 4 * 99]):
        p2, s2, c2 = _grads([100, 50], at)
        assert clip(p=p2, s=s2, c=c2) == -4
    assert clip(o=P + 4 * 99) == -4
    assert clip(o=P + 4 * 1000 + 1) == -3
    assert lib.qlora_grad_workspace_bytes(None, 2) == 0 and lib.qlora_grad_workspace_bytes(num, -1) == 0


def _int8(n=8, k=100, ld=128):
    return B.PackedInt8(n, k, torch.zeros(n, ld, dtype=torch.int8), torch.zeros(n))


def test_binding_rejects_rows():
    x = torch.zeros(4, 100, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="x must be bfloat16"):
        B.quantize_int8(x.double())
    with pytest.raises(ValueError, match="2-D"):
        B.quantize_int8(x[0])
    with pytest.raises(ValueError, match="2-D"):
        B.quantize_int8(x[:, :0])
    with pytest.raises(ValueError, match="contiguous"):
        B.quantize_int8(x[:, ::2])
    with pytest.raises(ValueError, match="out holds"):
        B.quantize_int8(x, out=_int8(5))
    with pytest.raises(ValueError, match="on the GPU"):
        B.quantize_int8(x)
    with pytest.raises(TypeError, match="dtype must be"):
        B.dequantize_int8(_int8(), torch.int8)
    with pytest.raises(ValueError, match="out has shape"):
        B.dequantize_int8(_int8(), out=torch.zeros(8, 128, dtype=torch.bfloat16))


def test_binding_rejects_packed_int8():
    for bad, err in ((_int8(ld=100), ValueError), (_int8(k=129), ValueError), (_int8(k=0), ValueError),
                     (B.PackedInt8(9, 100, torch.zeros(8, 128, dtype=torch.int8), torch.zeros(8)), ValueError),
                     (B.PackedInt8(8, 100, torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(8)), TypeError),
                     (B.PackedInt8(8, 100, torch.zeros(8, 128, dtype=torch.int8), torch.zeros(7)), ValueError),
                     (B.PackedInt8(8, 100, torch.zeros(8, 128, dtype=torch.int8), torch.zeros(8).double()), TypeError),
                     (B.PackedInt8(8, 100, torch.zeros(128, 8, dtype=torch.int8).t(), torch.zeros(8)), ValueError)):
        with pytest.raises(err):
            B.dequantize_int8(bad)
        with pytest.raises(err):
            B.int8_linear_fwd(bad, _int8())
    with pytest.raises(ValueError, match="rows of"):
        B.int8_linear_fwd(_int8(), _int8(k=99))
    with pytest.raises(ValueError, match="padded to the same length"):
        B.int8_linear_fwd(_int8(), _int8(ld=192))
    with pytest.raises(ValueError, match="out has shape"):
        B.int8_linear_fwd(_int8(), _int8(3), out=torch.zeros(8, 3, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="dtype must be"):
        B.int8_linear_fwd(_int8(), _int8(3), torch.float64)


def test_binding_rejects_norm_tensors():
    x = torch.zeros(4, 100, dtype=torch.bfloat16)
    g = torch.ones(100, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="gain has dtype"):
        B.rmsnorm_int8(x, g.half())
    with pytest.raises(ValueError, match="gain must be"):
        B.rmsnorm_int8(x, g[:99])
    with pytest.raises(TypeError, match="residual has dtype"):
        B.rmsnorm_int8(x, g, residual=x.float())
    with pytest.raises(ValueError, match="residual must be"):
        B.rmsnorm_int8(x, g, residual=x[:2])
    with pytest.raises(ValueError, match="residual_out must be"):
        B.rmsnorm_int8(x, g, residual=x, residual_out=torch.zeros(100, 4, dtype=torch.bfloat16).t())
    with pytest.raises(ValueError, match="without a residual"):
        B.rmsnorm_int8(x, g, residual_out=x)
    with pytest.raises(ValueError, match="out holds"):
        B.rmsnorm_int8(x, g, out=_int8(4, 99))


def test_binding_rejects_gradients():
    a, b = torch.zeros(10), torch.zeros(4, 5)
    with pytest.raises(TypeError, match="must be bfloat16"):
        B.GradList([a.double()])
    with pytest.raises(TypeError, match="gradient 1 has dtype"):
        B.GradList([a, b.half()])
    with pytest.raises(ValueError, match="gradient 1 must be contiguous"):
        B.GradList([a, b.t()])
    with pytest.raises(ValueError, match="out has shape"):
        B.grad_clip([a, b], 1.0, out=torch.zeros(29))
    with pytest.raises(ValueError, match="norm must be"):
        B.grad_clip([a, b], 1.0, norm=torch.zeros(2))
    with pytest.raises(ValueError, match="ws must be"):
        B.grad_norm([a, b], ws=torch.zeros(4))
    with pytest.raises(ValueError, match="on the GPU"):
        B.grad_norm([a, b])
