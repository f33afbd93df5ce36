"""GPU parity of the 8-bit rows, the norm that makes them and their product.

Codes, scales of quantized rows, values and products are bit-equal to the
oracle's: the codes are the exact rounding of 127 v / a (v one float32 value,
formed in the same order), scales and values are single float32 roundings, and
the product's sums are exact integers. The norm's scale takes a 64-bit sum
whose order differs from the oracle's: relative difference at most about
cols 2^-53, so the two float32 roundings differ by at most one step, 2^-23."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import int8 as OI

pytestmark = pytest.mark.gpu

TYPES = ("bfloat16", "float16", "float32")


def _t(name):
    import torch

    return getattr(torch, name)


def _rows(rows, cols, dtype, seed, spread=True):
    """Seeded rows of the type, each with a size of its own; exact ties in the
    first (its largest value is 4, half of that is 63.5 steps)."""
    import torch

    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols)) * (10.0 ** rng.uniform(-2, 2, (rows, 1)) if spread else 1.0)
    if rows and cols > 3:
        v[0] = np.clip(np.rint(v[0] * 4) / 4, -4, 4)
        v[0, :3] = (4.0, 2.0, -2.0)
    return torch.from_numpy(v.astype(np.float32)).to(_t(dtype))


def _same(got, want):
    """Bit-equal float arrays (any NaN equals any NaN)."""
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(np.where(nan, 0, got).view(np.uint32), np.where(nan, 0, want).view(np.uint32))


def _f32(t):
    return t.detach().float().cpu().numpy()


def _round(v, dtype):
    """float32 numpy values rounded to a torch type, as float32 again."""
    import torch

    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(_t(dtype)).float().numpy()


# rows x cols: one element, under and over a vector, odd widths, whole 64s, wide rows, many short rows
SHAPES = [(1, 1), (3, 7), (2, 64), (5, 65), (4, 200), (33, 515), (1, 4096), (3, 5001), (2, 8192), (2, 11008),
          (2, 22016), (1, 40001), (700, 16), (300, 129)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_rows_bit_exact(gpu_lib, shape, dtype):
    import torch

    rows, cols = shape
    say(f"[int8 rows] {rows}x{cols} {dtype}")
    x = _rows(rows, cols, dtype, 11 * rows + cols)
    q = gpu_lib.quantize_int8(x.cuda())
    torch.cuda.synchronize()
    codes, scale = OI.quantize(x.float().numpy())
    got = q.codes.cpu().numpy()
    assert got.shape == (rows, -(-cols // 64) * 64)
    assert np.array_equal(got[:, :cols], codes)
    assert not got[:, cols:].any()
    _same(q.scale.cpu().numpy(), scale)
    for out in TYPES:
        v = gpu_lib.dequantize_int8(q, _t(out))
        _same(_f32(v), _round(OI.dequantize(codes, scale), out))


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_special_values(gpu_lib, dtype):
    """Rows of zeros, with NaN, with infinities, of the type's largest and
    smallest values; their neighbours keep their results."""
    import torch

    fi = torch.finfo(_t(dtype))
    x = _rows(10, 100, dtype, 5)
    x[1] = 0
    x[2, 99] = float("nan")
    x[4, 0] = float("inf")
    x[5, 50] = float("-inf")
    x[6] = fi.max * torch.sign(x[6])
    x[7] = fi.tiny
    x[8] = 0
    x[8, 17] = fi.smallest_normal / 2 if dtype != "float32" else 1e-44  # a subnormal
    codes, scale = OI.quantize(x.float().numpy())
    assert np.isnan(scale[[2, 4, 5]]).all()
    say(f"[int8 rows] special values {dtype}")
    q = gpu_lib.quantize_int8(x.cuda())
    v = gpu_lib.dequantize_int8(q, torch.float32)
    torch.cuda.synchronize()
    assert np.array_equal(q.codes.cpu().numpy()[:, :100], codes)
    _same(q.scale.cpu().numpy(), scale)
    _same(v.cpu().numpy(), OI.dequantize(codes, scale))


def _scale_close(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.all(np.abs(got[ok].astype(np.float64) - want[ok]) <= 2.0 ** -23 * np.abs(want[ok]))


@pytest.mark.parametrize("dtype,gain_type", [(t, g) for t in TYPES for g in dict.fromkeys((t, "float32"))])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("with_residual", [True, False], ids=["residual", "plain"])
def test_rmsnorm_bit_exact(gpu_lib, shape, dtype, gain_type, with_residual):
    import torch

    rows, cols = shape
    say(f"[rmsnorm int8] {rows}x{cols} {dtype} gain {gain_type} residual {with_residual}")
    x = _rows(rows, cols, dtype, 3 * rows + cols)
    r = _rows(rows, cols, dtype, 5 * rows + cols) if with_residual else None
    gain = (1 + 0.2 * torch.from_numpy(np.random.default_rng(cols).standard_normal(cols))).to(_t(gain_type))
    q, h = gpu_lib.rmsnorm_int8(x.cuda(), gain.cuda(), 1e-5, residual=None if r is None else r.cuda())
    torch.cuda.synchronize()
    codes, scale, href = OI.rmsnorm(x.float().numpy(), gain.float().numpy(), 1e-5,
                                    None if r is None else r.float().numpy())
    got = q.codes.cpu().numpy()
    assert np.array_equal(got[:, :cols], codes)
    assert not got[:, cols:].any()
    _scale_close(q.scale.cpu().numpy(), scale)
    if with_residual:
        _same(_f32(h), _round(href, dtype))
    else:
        assert h is None


@pytest.mark.parametrize("into", ["residual", "x"])
@pytest.mark.parametrize("shape", [(3, 500), (2, 4096), (1, 40001)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_rmsnorm_in_place(gpu_lib, shape, into):
    import torch

    rows, cols = shape
    x, r = _rows(rows, cols, "bfloat16", 1).cuda(), _rows(rows, cols, "bfloat16", 2).cuda()
    gain = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    say(f"[rmsnorm int8] {rows}x{cols} in place of {into}")
    q0, h0 = gpu_lib.rmsnorm_int8(x, gain, residual=r)
    q1, h1 = gpu_lib.rmsnorm_int8(x, gain, residual=r, residual_out=r if into == "residual" else x, out=q0.__class__(
        rows, cols, torch.full_like(q0.codes, 55), torch.empty_like(q0.scale)))
    torch.cuda.synchronize()
    assert h1 is (r if into == "residual" else x)
    assert torch.equal(h0, h1) and torch.equal(q0.codes, q1.codes) and torch.equal(q0.scale, q1.scale)


def test_rmsnorm_special_rows(gpu_lib):
    """Zeros with eps = 0, NaN, infinities, magnitudes whose squares pass
    float32's range in both directions, and a gain that is zero or not finite."""
    import torch

    x = _rows(8, 130, "float32", 9)
    x[1] = 0
    x[2, 129] = float("nan")
    x[3, 0] = float("-inf")
    x[4] *= 1e25
    x[5] *= 1e-30
    gain = torch.ones(130)
    gain[7] = 0
    say("[rmsnorm int8] special rows")
    for bad in (None, float("inf"), float("nan")):
        if bad is not None:
            gain[9] = bad
        q, _ = gpu_lib.rmsnorm_int8(x.cuda(), gain.cuda(), 0.0)
        torch.cuda.synchronize()
        codes, scale, _ = OI.rmsnorm(x.numpy(), gain.numpy(), 0.0)
        assert np.array_equal(q.codes.cpu().numpy()[:, :130], codes)
        _scale_close(q.scale.cpu().numpy(), scale)
        if bad is None:
            assert np.isnan(scale[[2, 3]]).all() and np.isfinite(scale[[0, 1, 4, 5, 6, 7]]).all() and scale[4] > 0


def _operands(m, n, k, seed, full=False):
    """Codes (padded to 64) and scales; full: every code at the ends of the range."""
    rng = np.random.default_rng(seed)
    ld = -(-k // 64) * 64

    def one(rows):
        c = np.zeros((rows, ld), np.int8)
        c[:, :k] = rng.choice([-128, 127], (rows, k)) if full else np.clip(np.rint(rng.standard_normal((rows, k)) * 32),
                                                                         -127, 127)
        return c, (10.0 ** rng.uniform(-3, -1, rows)).astype(np.float32)

    return one(n) + one(m)


def _packed(gpu_lib, codes, scale, k):
    import torch

    return gpu_lib.PackedInt8(codes.shape[0], k, torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda())


# m, n, k: decode sizes, the edges of every tile and of the split along k, odd sizes, whole tiles
LINEAR = [(1, 1, 1), (1, 16, 64), (1, 257, 4096), (2, 33, 100), (3, 4096, 64), (8, 130, 11008), (15, 48, 192),
          (16, 512, 4096), (17, 100, 320), (31, 1000, 1024), (32, 64, 4160), (33, 129, 128), (48, 2048, 512),
          (63, 65, 64), (64, 256, 22016), (65, 300, 640), (100, 1009, 777), (127, 255, 4096), (128, 128, 128),
          (129, 513, 192), (200, 4097, 448), (256, 256, 1088), (257, 511, 2112), (300, 5003, 320), (512, 1024, 4096),
          (1000, 777, 1000), (1025, 130, 64), (2048, 256, 256)]


@pytest.mark.parametrize("size", LINEAR, ids=lambda s: "x".join(map(str, s)))
def test_linear_bit_exact(gpu_lib, size):
    import torch

    m, n, k = size
    say(f"[int8 linear] m={m} n={n} k={k}")
    w, sw, x, sx = _operands(m, n, k, m + 3 * n + 7 * k)
    want = OI.linear(w, sw, x, sx)
    qw, qx = _packed(gpu_lib, w, sw, k), _packed(gpu_lib, x, sx, k)
    for dtype in TYPES:
        y = torch.full((m, n), 7.0, dtype=_t(dtype), device="cuda")
        assert gpu_lib.int8_linear_fwd(qw, qx, _t(dtype), out=y) is y
        torch.cuda.synchronize()
        _same(_f32(y), _round(want, dtype))


# Larger sizes, for which each of the tiles is the cheapest; contractions that end
# in the middle of a unit of 128 codes and leave every remainder of the ring.
TILES = [(m, n, k) for m, n, ks in (
    (1604, 5012, (64, 128, 192)), (2317, 3460, (640, 832, 1088, 1216, 1472, 1536)),    # 256 x 256
    (1282, 3848, (64, 128, 192)), (776, 5012, (832, 960, 1088, 1536)),                 # 128 x 256
    (592, 4915, (64, 128)), (385, 4721, (192, 320, 832, 960, 1088, 1472, 1536)),       # 128 x 128
    (201, 4139, (192, 320, 832, 960, 1088, 1536)),                                     # 64 x 128
    (2064, 65, (64, 128, 832, 1088, 1472, 1536, 2112)), (1650, 259, (960, 1472, 1536)),  # 64 x 64, 32 x 64
) for k in ks]


@pytest.mark.parametrize("size", TILES, ids=lambda s: "x".join(map(str, s)))
def test_linear_every_tile(gpu_lib, size):
    import torch

    m, n, k = size
    say(f"[int8 linear] tiles m={m} n={n} k={k}")
    w, sw, x, sx = _operands(m, n, k, m + 3 * n + 7 * k)
    want = OI.linear(w, sw, x, sx)
    qw, qx = _packed(gpu_lib, w, sw, k), _packed(gpu_lib, x, sx, k)
    for dtype in ("bfloat16", "float32"):
        y = torch.full((m, n), 7.0, dtype=_t(dtype), device="cuda")
        gpu_lib.int8_linear_fwd(qw, qx, _t(dtype), out=y)
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), torch.from_numpy(want).to(_t(dtype)))


@pytest.mark.parametrize("m", [1, 16, 70, 300])
def test_linear_largest_sums(gpu_lib, m):
    """Codes of -128 and 127 alone at the longest k: the sums come within 1.1%
    of 2^31 where a row meets itself, and must not wrap."""
    import torch

    n, k = 40, 131008
    say(f"[int8 linear] largest sums m={m}")
    w, sw, x, sx = _operands(m, n, k, m, full=True)
    w[0], x[0] = -128, -128
    y = gpu_lib.int8_linear_fwd(_packed(gpu_lib, w, sw, k), _packed(gpu_lib, x, sx, k), torch.float32)
    torch.cuda.synchronize()
    want = OI.linear(w, sw, x, sx)
    _same(y.cpu().numpy(), want)
    assert want[0, 0] == np.float32(np.float32(128 * 128 * k) * sx[0]) * sw[0]


def test_linear_scales_not_finite_and_zero(gpu_lib):
    """A token or channel with scale NaN gives a row or column of NaN and
    leaves the others; scale 0 gives zeros; large scales overflow to infinity."""
    import torch

    for m in (2, 40, 300):
        n, k = 100, 256
        say(f"[int8 linear] special scales m={m}")
        w, sw, x, sx = _operands(m, n, k, m)
        sx[1], sw[5], sw[6], sw[7] = np.nan, np.nan, 0.0, 3e38
        for dtype in TYPES:
            y = gpu_lib.int8_linear_fwd(_packed(gpu_lib, w, sw, k), _packed(gpu_lib, x, sx, k), _t(dtype))
            torch.cuda.synchronize()
            _same(_f32(y), _round(OI.linear(w, sw, x, sx), dtype))


def test_linear_token_rows_do_not_depend_on_m(gpu_lib):
    """A token's row is bit-identical alone, in a small batch and in a large one."""
    import torch

    n, k = 1111, 4160
    w, sw, x, sx = _operands(600, n, k, 3)
    qw = _packed(gpu_lib, w, sw, k)
    say("[int8 linear] the same token at every m")
    whole = gpu_lib.int8_linear_fwd(qw, _packed(gpu_lib, x, sx, k), torch.float32)
    for m in (1, 2, 5, 16, 17, 33, 64, 65, 128, 200, 400):
        part = gpu_lib.int8_linear_fwd(qw, _packed(gpu_lib, x[:m].copy(), sx[:m].copy(), k), torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(part, whole[:m]), m


def test_linear_in_two_launches(gpu_lib):
    """A size whose 256 x 256 tiles fill three rounds of the CUs and part of a
    fourth, whose channels go to two launches: every token's row is bit-equal to
    the one computed in batches of 50, and sampled rows to the oracle's."""
    import torch

    m, n, k = 1000, 53248 + 77, 1856
    say(f"[int8 linear] two launches, m={m} n={n} k={k}")
    rng = np.random.default_rng(4)
    w, sw, _, _ = _operands(1, n, k, 5)
    x = np.clip(np.rint(rng.standard_normal((m, k)) * 32), -127, 127).astype(np.int8)
    sx = (10.0 ** rng.uniform(-3, -1, m)).astype(np.float32)
    qw = _packed(gpu_lib, w, sw, k)
    for dtype in ("bfloat16", "float32"):
        y = gpu_lib.int8_linear_fwd(qw, _packed(gpu_lib, x, sx, k), _t(dtype))
        for a in range(0, m, 50):
            part = gpu_lib.int8_linear_fwd(qw, _packed(gpu_lib, x[a:a + 50], sx[a:a + 50], k), _t(dtype))
            torch.cuda.synchronize()
            assert torch.equal(y[a:a + 50], part)
        pick = [0, 255, 256, 511, 767, 768, 999]
        _same(_f32(y[pick]), _round(OI.linear(w, sw, x[pick], sx[pick]), dtype))


@pytest.mark.parametrize("m", [1, 40, 300])
def test_writes_stay_inside(gpu_lib, m):
    """Memory behind the outputs keeps its values (odd sizes)."""
    import torch

    n, k = 1003, 323
    say(f"[int8] nothing behind the outputs is written, m={m}")
    w, sw, x, sx = _operands(m, n, k, 8)
    buf = torch.full((m * n + 512,), 9.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.int8_linear_fwd(_packed(gpu_lib, w, sw, k), _packed(gpu_lib, x, sx, k), out=buf[:m * n].view(m, n))
    xb = _rows(m, k, "bfloat16", 4).cuda()
    ld = 384
    codes = torch.full((m * ld + 512,), 9, dtype=torch.int8, device="cuda")
    scale = torch.full((m + 64,), 9.0, device="cuda")
    q = gpu_lib.PackedInt8(m, k, codes[:m * ld].view(m, ld), scale[:m])
    gpu_lib.quantize_int8(xb, out=q)
    vals = torch.full((m * k + 512,), 9.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.dequantize_int8(q, out=vals[:m * k].view(m, k))
    hbuf = torch.full((m * k + 512,), 9.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.rmsnorm_int8(xb, torch.ones(k, device="cuda"), residual=xb, residual_out=hbuf[:m * k].view(m, k), out=q)
    torch.cuda.synchronize()
    for t, used in ((buf, m * n), (codes, m * ld), (scale, m), (vals, m * k), (hbuf, m * k)):
        assert (t[used:] == 9).all()
    assert not codes[:m * ld].view(m, ld)[:, k:].any()


@pytest.mark.parametrize("m", [1, 24, 130])
def test_serving_chain_in_a_graph(gpu_lib, m):
    """Norm -> product -> quantize -> product, as a layer's first half runs,
    captured once and replayed on new inputs: every replay equals the eager
    calls. Two graphs captured from the same code share no workspace."""
    import torch

    k, n = 1024, 777
    rng = np.random.default_rng(2)
    w1 = gpu_lib.quantize_int8(torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)).cuda())
    w2 = gpu_lib.quantize_int8(torch.from_numpy(rng.standard_normal((300, n)).astype(np.float32)).cuda())
    gain = torch.ones(k, dtype=torch.bfloat16, device="cuda")

    def chain(x, r):
        q, h = gpu_lib.rmsnorm_int8(x, gain, residual=r)
        mid = gpu_lib.int8_linear_fwd(w1, q)
        return gpu_lib.int8_linear_fwd(w2, gpu_lib.quantize_int8(mid), torch.float32), h

    x = [_rows(m, k, "bfloat16", i, spread=False).cuda() for i in range(2)]
    r = [_rows(m, k, "bfloat16", 10 + i, spread=False).cuda() for i in range(2)]
    say(f"[int8] chain in graphs, m={m}")
    chain(x[0], r[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain(x[i], r[i]))
        graphs.append(g)
    for step in range(3):
        for i in range(2):
            x[i].copy_(_rows(m, k, "bfloat16", 20 + 2 * step + i, spread=False))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] for o in outs]
        for i in range(2):
            want = chain(x[i], r[i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got[i], want))


def test_merged_adapter_served_in_8_bits(gpu_lib):
    """The way of an adapter: trained layer -> merged weight -> 8-bit rows ->
    the norm's 8-bit output through the product, against the float64 product of
    the merged weight and the normed input.

    Tolerance, of the root of the mean square: a code is off by at most half a
    step, uniformly: error step / sqrt(12) each. The step is max / 127, and a
    row of 512 normals has max about 3.2 sigma (at most 4.5), so each side's
    relative error is at most 4.5 / 127 / sqrt(12) = 1.03%, both sides 1.45%;
    the merged weight's and Y's bf16 roundings add 2^-9 each: 1.6% bounds it."""
    import torch

    from gpu_cases import layer_inputs

    n, k, m, r, alpha = 320, 512, 48, 8, 16.0
    w, x, a, b, _ = layer_inputs(n, k, m, r, "int8_served")
    q = gpu_lib.quantize(torch.from_numpy(w).cuda())
    merged = gpu_lib.merge(q, a.cuda(), b.cuda(), alpha, torch.float32)
    gain = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    say("[int8] merged adapter served in 8 bits")
    served = gpu_lib.quantize_int8(merged)
    qx, _ = gpu_lib.rmsnorm_int8(x.cuda(), gain, 1e-6)
    y = gpu_lib.int8_linear_fwd(served, qx)
    torch.cuda.synchronize()
    xn = x.double().numpy()
    xn = xn / np.sqrt((xn ** 2).mean(axis=1, keepdims=True) + 1e-6)
    want = xn @ merged.double().cpu().numpy().T
    err = np.sqrt(np.mean((_f32(y) - want) ** 2) / np.mean(want ** 2))
    say(f"   relative error {err:.4f}")
    assert err <= 0.016


def test_life_of_an_adapter(gpu_lib):
    """One training step with clipped gradients, the merge, and serving in 8
    bits: the calls of both ends together. The step's update is checked against
    float64, and the served output as in the test above (its 1.6%, and the
    update's float32 roundings, far below it)."""
    import torch

    from gpu_cases import layer_inputs

    n, k, m, r, alpha, lr = 256, 512, 40, 8, 16.0, 0.05
    w, x, a, b, dy = layer_inputs(n, k, m, r, "life_of_an_adapter")
    q = gpu_lib.quantize(torch.from_numpy(w).cuda())
    x, a, b, dy = x.cuda(), a.cuda(), b.cuda(), dy.cuda()
    say("[int8] life of an adapter")
    _, h = gpu_lib.linear_fwd(q, x, a, b, alpha)
    _, da, db = gpu_lib.linear_bwd(q, x, dy, a, b, alpha, h=h)
    raw = [da.double(), db.double()]
    norm = gpu_lib.grad_clip([da, db], 1.0)
    torch.cuda.synchronize()
    total = sum(float(g.square().sum()) for g in raw) ** 0.5
    assert total > 1.0 and abs(float(norm) - total) <= 2.0 ** -22 * total
    for g, c in zip(raw, (da, db)):
        # the factor's and the product's roundings
        assert ((c.double() - g / (total + 1e-6)).abs() <= 2.0 ** -22 * (g / total).abs()).all()
    a2, b2 = (a.float() - lr * da).bfloat16(), (b.float() - lr * db).bfloat16()
    merged = gpu_lib.merge(q, a2, b2, alpha, torch.float32)
    served = gpu_lib.quantize_int8(merged)
    res = x.clone()
    qx, hid = gpu_lib.rmsnorm_int8(dy[:, :n].repeat(1, k // n), torch.ones(k, device="cuda"), 1e-6, residual=res,
                                   residual_out=res)
    y = gpu_lib.int8_linear_fwd(served, qx)
    torch.cuda.synchronize()
    assert hid is res
    hn = (x.double() + dy.double().repeat(1, k // n)).cpu().numpy()
    hn = hn / np.sqrt((hn ** 2).mean(axis=1, keepdims=True) + 1e-6)
    want = hn @ merged.double().cpu().numpy().T
    err = np.sqrt(np.mean((_f32(y) - want) ** 2) / np.mean(want ** 2))
    say(f"   relative error {err:.4f}")
    assert err <= 0.016


def test_other_stream(gpu_lib):
    """Calls run on the caller's current stream."""
    import torch

    w, sw, x, sx = _operands(20, 64, 128, 1)
    qw, qx = _packed(gpu_lib, w, sw, 128), _packed(gpu_lib, x, sx, 128)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = gpu_lib.int8_linear_fwd(qw, qx, torch.float32)
    s.synchronize()
    _same(y.cpu().numpy(), OI.linear(w, sw, x, sx))


def test_no_rows_and_no_tokens(gpu_lib):
    import torch

    for dtype in TYPES:
        x = torch.empty((0, 70), dtype=_t(dtype), device="cuda")
        q = gpu_lib.quantize_int8(x)
        assert q.codes.shape == (0, 128) and q.scale.shape == (0,)
        assert gpu_lib.dequantize_int8(q, _t(dtype)).shape == (0, 70)
        qn, h = gpu_lib.rmsnorm_int8(x, torch.ones(70, device="cuda"), residual=x)
        assert qn.n == 0 and h.shape == (0, 70)
        w, sw, _, _ = _operands(1, 9, 70, 1)
        assert gpu_lib.int8_linear_fwd(_packed(gpu_lib, w, sw, 70), q, _t(dtype)).shape == (0, 9)


def test_another_current_device(gpu_lib, monkeypatch):
    """Where the tensors' GPU is not the current one the call makes it so: with
    one GPU, the current index is read as another."""
    w, sw, x, sx = _operands(20, 64, 128, 1)
    qw, qx = _packed(gpu_lib, w, sw, 128), _packed(gpu_lib, x, sx, 128)
    gpu_lib.int8_linear_fwd(qw, qx)
    monkeypatch.setattr(gpu_lib, "_device_now", lambda: 1)
    import torch

    y = gpu_lib.int8_linear_fwd(qw, qx, torch.float32)
    torch.cuda.synchronize()
    _same(y.cpu().numpy(), OI.linear(w, sw, x, sx))


def test_two_streams_at_once(gpu_lib):
    """Calls of the same shapes on two streams, each on its own buffers: no
    state is shared between them."""
    import torch

    n, k = 777, 1024
    rng = np.random.default_rng(8)
    qw = gpu_lib.quantize_int8(torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)).cuda())
    xs = [_rows(200, k, "bfloat16", i, spread=False).cuda() for i in range(2)]
    gain = torch.ones(k, device="cuda")
    grads = [[torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda() for s in (5000, 70001)] for _ in range(2)]

    def work(i):
        q, h = gpu_lib.rmsnorm_int8(xs[i], gain, residual=xs[1 - i])
        out = torch.empty(75001, device="cuda")
        norm = gpu_lib.grad_clip(grads[i], 1.0, out=out)
        return gpu_lib.int8_linear_fwd(qw, q), h, out, norm

    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
