"""Outputs of the 8-bit row calls that overlap an input or another output are
refused before any launch (no GPU: fake aligned addresses, and every call here
is refused). One workgroup's writes would change what another still has to
read."""
import pytest

from bit_nf4_quantized_18_amd import binding as B

BF16, F32, F16 = B.QLORA_BF16, B.QLORA_F32, B.QLORA_F16
ROWS, COLS, LD = 40, 100, 128
X, RES, GAIN, OUT, CODES, SCALE = (i << 20 for i in range(1, 7))
SIZE = {BF16: 2, F16: 2, F32: 4}


def _bytes(t):
    return ROWS * COLS * SIZE[t]


def _around(at, bytes_, mine):
    """Addresses (16-byte steps) at which `mine` bytes meet the buffer [at, at + bytes_)."""
    return [at, at + 16, at + (bytes_ - 1) // 16 * 16, at - 16, at - (mine - 1) // 16 * 16]


@pytest.mark.parametrize("t", [BF16, F32, F16])
def test_quantize_and_dequantize(t):
    lib = B.load()

    def q(x=X, codes=CODES, scale=SCALE):
        return lib.qlora_int8_quantize(x, t, ROWS, COLS, codes, LD, scale, None)

    def d(codes=CODES, scale=SCALE, out=OUT):
        return lib.qlora_int8_dequantize(codes, LD, scale, ROWS, COLS, t, out, None)

    assert all(q(codes=a) == -4 for a in _around(X, _bytes(t), ROWS * LD))
    assert all(q(scale=a) == -4 for a in _around(X, _bytes(t), ROWS * 4))
    assert all(q(scale=a) == -4 for a in _around(CODES, ROWS * LD, ROWS * 4))
    assert all(d(out=a) == -4 for a in _around(CODES, ROWS * LD, _bytes(t)))
    assert all(d(out=a) == -4 for a in _around(SCALE, ROWS * 4, _bytes(t)))


@pytest.mark.parametrize("t,gt", [(BF16, BF16), (BF16, F32), (F16, F16), (F32, F32)])
def test_rmsnorm(t, gt):
    lib = B.load()

    def f(x=X, res=RES, gain=GAIN, out=OUT, codes=CODES, scale=SCALE):
        return lib.qlora_rmsnorm_int8(x, res, gain, t, gt, ROWS, COLS, 1e-6, out, codes, LD, scale, None)

    n = _bytes(t)
    for at in (X, RES):
        # shifted over an input; its own place alone is taken
        assert all(f(out=a) == -4 for a in _around(at, n, n) if a != at)
    # in the place of one input, while the other is a shifted view of it
    assert f(x=RES + 64, out=RES) == -4 and f(res=X + 64, out=X) == -4
    assert all(f(out=a) == -4 for a in _around(GAIN, COLS * SIZE[gt], n))
    for at, size in ((X, n), (RES, n), (GAIN, COLS * SIZE[gt]), (OUT, n)):
        assert all(f(codes=a) == -4 for a in _around(at, size, ROWS * LD))
        assert all(f(scale=a) == -4 for a in _around(at, size, ROWS * 4))
    assert all(f(scale=a) == -4 for a in _around(CODES, ROWS * LD, ROWS * 4))
    # without a residual h is not written, its address does not count
    assert f(res=None, out=None, codes=X) == -4 and f(res=None, out=X, scale=GAIN) == -4


@pytest.mark.parametrize("over", ["w_codes", "w_scale", "x_codes", "x_scale"])
def test_product_output(over):
    """The binding refuses an output over the operands (CPU tensors: an output
    behind them is refused for these, later)."""
    import torch

    m, n, k = 8, 64, 64
    pool = torch.zeros(1 << 16, dtype=torch.uint8)
    at = {"w_codes": (0, n * k), "w_scale": (8192, n * 4), "x_codes": (16384, m * k), "x_scale": (24576, m * 4)}
    part = {name: pool[a:a + b] for name, (a, b) in at.items()}
    w = B.PackedInt8(n, k, part["w_codes"].view(torch.int8).view(n, k), part["w_scale"].view(torch.float32))
    x = B.PackedInt8(m, k, part["x_codes"].view(torch.int8).view(m, k), part["x_scale"].view(torch.float32))
    a, b = at[over]
    size = m * n * 2
    name = {"w": "the weight's ", "x": "x's "}[over[0]] + over[2:]
    place = lambda i: pool[i:i + size].view(torch.bfloat16).view(m, n)  # noqa: E731
    for i in [a, a + b - 16] + ([a - size + 16] if a >= size else []):
        with pytest.raises(ValueError, match="out overlaps " + name):
            B.int8_linear_fwd(w, x, out=place(i))
    with pytest.raises(ValueError, match="on the GPU"):
        B.int8_linear_fwd(w, x, out=place(a + b))
