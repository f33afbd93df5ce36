"""The operators of a gated feed-forward block together, as a training step and as a served model use them.

Training: forward of the block and of its down projection; of the activations only 8-bit rows are kept; backward
through both. Serving: norm and rounding to 8 bits, the block and the down projection in 8-bit integers."""
import numpy as np
import pytest
import torch

import gated_cases as C
import test_gpu_linear_x8 as X
from oracle import gated as OG

pytestmark = pytest.mark.gpu

K, HALF, R, T = 320, 512, 16, torch.bfloat16
S = 2.0  # alpha / r


class Layer:
    """Weights and an input on the GPU, and the same numbers in float64 here."""

    def __init__(self, lib, m, seed):
        draw = lambda shape, std, i: C.normal(shape, std, seed + i).to(T).cuda()  # noqa: E731
        self.lib, self.m = lib, m
        self.wg = lib.quantize(C.normal((2 * HALF, K), 1.5 / K ** 0.5, seed).float().cuda())
        self.wd = lib.quantize(C.normal((K, HALF), 1.0 / HALF ** 0.5, seed + 1).float().cuda())
        self.ag, self.bg = draw((2 * R, K), 1 / R, 2), draw((2 * HALF, R), 0.05, 3)
        self.ad, self.bd = draw((R, HALF), 1 / R, 4), draw((K, R), 0.05, 5)
        self.x, self.do = draw((m, K), 1.0, 6), draw((m, K), 1.0, 7)
        self.wg64, self.wd64 = (lib.dequantize(w, T).cpu().double() for w in (self.wg, self.wd))
        self.f64 = {n: getattr(self, n).cpu().double() for n in ("x", "ag", "bg", "ad", "bd", "do")}

    def forward(self, act):
        """(output, what the backward keeps: 8-bit rows of x, of [G | U] and of P, and both H)."""
        lib = self.lib
        p, y, h = lib.linear_fwd_gated(self.wg, self.x, self.ag, self.bg, S * R, act)
        out, hd = lib.linear_fwd(self.wd, p, self.ad, self.bd, S * R)
        return out, (lib.quantize_int8(self.x), lib.quantize_int8(y.view(2 * self.m, HALF)), lib.quantize_int8(p), h, hd)

    def backward(self, act, kept, do):
        lib, (x8, y8, p8, h, hd) = self.lib, kept
        dp, dad, dbd = lib.linear_bwd(self.wd, p8, do, self.ad, self.bd, S * R, h=hd)
        dy = lib.gated_bwd(y8, dp, act)
        dx, dag, dbg = lib.linear_bwd_grouped(self.wg, [HALF, HALF], x8, dy, self.ag, self.bg, S * R, h=h)
        return dp, dy, {"x": dx, "ag": dag, "bg": dbg, "ad": dad, "bd": dbd}

    def exact(self, act, **other):
        """The block in float64: every intermediate; `other` replaces inputs."""
        v = {**self.f64, **other}
        mm = lambda p, q: p @ q.t().contiguous()  # noqa: E731
        h = mm(v["x"], v["ag"])
        y = mm(v["x"], self.wg64) + S * torch.cat([mm(h[:, l * R:(l + 1) * R], v["bg"][l * HALF:(l + 1) * HALF])
                                                    for l in range(2)], 1)
        p = torch.from_numpy(OG.fwd(y[:, :HALF].numpy(), y[:, HALF:].numpy(), act))
        hd = mm(p, v["ad"])
        return h, y, p, hd, mm(p, self.wd64) + S * mm(hd, v["bd"])


def kept64(kept, m):
    """The checkpoints' values in float64."""
    value = lambda q: q.codes[:, :q.k].cpu().double() * q.scale.cpu().double()[:, None]  # noqa: E731
    x8, y8, p8, h, hd = kept
    return value(x8), value(y8).view(m, 2 * HALF), value(p8), h.cpu().double(), hd.cpu().double()


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("m", [3, 48, 301])
def test_each_link_of_a_training_step(gpu_lib, m, act):
    v = Layer(gpu_lib, m, 40 + m)
    _, kept = v.forward(act)
    x8, _, p8, h, hd = kept
    kx, ky, _, _, _ = kept64(kept, m)
    # 8-bit rows: half a step of absmax / 127 (and the float32 scale's rounding) from the value that was rounded
    x64 = v.f64["x"]
    assert ((kx - x64).abs() <= x64.abs().amax(1, keepdim=True) / 254 * 1.0001).all()
    dp, dy, grads = v.backward(act, kept, v.do)
    down = X.expected(gpu_lib, v.wd, p8, v.do, hd, v.ad, v.bd, S * R, 1, T)
    for name, got, (want, off) in zip(("dP", "dA down", "dB down"), (dp, grads["ad"], grads["bd"]), down):
        C.check(got, want, off, name)
    g, u, d = ky[:, :HALF].numpy(), ky[:, HALF:].numpy(), C.f64(dp)
    # the rows' float32 products code x scale are half a step off, up to 1.2 times that in act' and act
    extra = 2 * C.F32 * np.abs(d) * (1 + np.abs(g)) * (1 + np.abs(u))
    for name, got, want, off in zip(("dG", "dU"), (dy[:, :HALF], dy[:, HALF:]), OG.bwd(g, u, d, act), C.bwd_bound(g, u, d, act, T)):
        C.check(got, want, off + extra, name)
    up = X.expected(gpu_lib, v.wg, x8, dy, h, v.ag, v.bg, S * R, 2, T)
    for name, got, (want, off) in zip(("dX", "dA", "dB"), (grads["x"], grads["ag"], grads["bg"]), up):
        C.check(got, want, off, name)


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("m", [5, 64])
def test_gradients_against_differences(gpu_lib, m, act):
    """Along the signs of a gradient the loss <dO, O> changes by the gradient's sum of magnitudes. The bounds follow each
    rounding (what the checkpoints are off is measured, what the kernels may be off is bounded) through the backward."""
    v = Layer(gpu_lib, m, 7 + m)
    _, kept = v.forward(act)
    dp, dy, grads = v.backward(act, kept, v.do)
    h64, y64, p64, hd64, _ = v.exact(act)
    kx, ky, kp, kh, khd = kept64(kept, m)
    mm = lambda p, q: p @ q.contiguous()  # noqa: E731
    f, do = v.f64, v.f64["do"]

    # down projection: dO and the weights are exact, P and H its checkpoints
    down = X.expected(gpu_lib, v.wd, kept[2], v.do, kept[4], v.ad, v.bd, S * R, 1, T)
    dhd = S * mm(do, f["bd"])
    dp64 = mm(do, v.wd64) + mm(dhd, f["ad"])
    dp_off = torch.from_numpy(down[0][1])

    # product: dG = dP U act'(G), dU = dP act(G) from the checkpoint of [G | U]
    fac = lambda y: [torch.from_numpy(q) for q in OG.bwd(y[:, :HALF].numpy(), y[:, HALF:].numpy(), 1.0, act)]  # noqa: E731
    dy64, dy_off = [], []
    for exact, stored, rounding in zip(fac(y64), fac(ky), C.bwd_bound(ky[:, :HALF].numpy(), ky[:, HALF:].numpy(),
                                                                      (dp64.abs() + dp_off).numpy(), act, T)):
        dy64.append(dp64 * exact)
        dy_off.append(dp64.abs() * (stored - exact).abs() + dp_off * stored.abs() + torch.from_numpy(rounding) * 1.01)
    dy64, dy_off = torch.cat(dy64, 1), torch.cat(dy_off, 1)

    # the block's projections
    up = X.expected(gpu_lib, v.wg, kept[0], dy, kept[3], v.ag, v.bg, S * R, 2, T)
    halves = [(slice(l * HALF, (l + 1) * HALF), slice(l * R, (l + 1) * R)) for l in range(2)]
    dh64 = torch.cat([S * mm(dy64[:, rows], f["bg"][rows]) for rows, _ in halves], 1)

    def error(name, way):
        """Bound of <gradient, way>'s error: what dY is off meets the change of [G | U] along `way` (from the checkpoints'
        values), what a checkpoint is off the other factor of its product, and the call's own roundings add up."""
        if name == "ad":
            return down[1][1].sum() + ((kp - p64) * mm(dhd, way)).sum().abs()
        if name == "bd":
            return down[2][1].sum() + S * ((khd - hd64) * mm(do, way)).sum().abs()
        if name == "x":
            ty = torch.cat([mm(way, v.wg64[rows].t()) + S * mm(mm(way, f["ag"][slots].t()), f["bg"][rows].t()) for rows, slots in halves], 1)
            return up[0][1].sum() + (dy_off * ty.abs()).sum()
        if name == "ag":
            ty = torch.cat([S * mm(mm(kx, way[slots].t()), f["bg"][rows].t()) for rows, slots in halves], 1)
            return up[1][1].sum() + (dy_off * ty.abs()).sum() + ((kx - f["x"]) * mm(dh64, way)).sum().abs()
        ty = torch.cat([S * mm(kh[:, slots], way[rows].t()) for rows, slots in halves], 1)
        other = sum((S * (kh - h64)[:, slots] * mm(dy64[:, rows], way[rows])).sum() for rows, slots in halves)
        return up[2][1].sum() + (dy_off * ty.abs()).sum() + other.abs()

    loss = lambda name, step: (do * v.exact(act, **{name: f[name] + step})[4]).sum()  # noqa: E731
    for name, grad in grads.items():
        grad = grad.cpu().double()
        way = torch.sign(grad)
        diff = [(loss(name, h * way) - loss(name, -h * way)) / (2 * h) for h in (2.0 ** -12, 2.0 ** -13)]
        got, tol = (grad * way).sum(), error(name, way) + 2 * (diff[0] - diff[1]).abs()
        print(f"{name}: {got:.6g}, differences {diff[1]:.6g}, bound {tol:.3g}")
        assert tol < 0.25 * got, "a bound that says nothing"
        assert (got - diff[1]).abs() <= tol, name


def test_training_step_captured_and_on_another_stream(gpu_lib):
    v = Layer(gpu_lib, 48, 3)
    out, kept = v.forward(OG.SILU)
    _, _, grads = v.backward(OG.SILU, kept, v.do)
    want = [out, *grads.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2, kept2 = v.forward(OG.SILU)
        got = [out2, *v.backward(OG.SILU, kept2, v.do)[2].values()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))

    # two graphs, each with the workspaces of its own memory pool, replayed in turn with eager calls between
    graphs, results = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, k = v.forward(OG.SILU)
            results.append([o, *v.backward(OG.SILU, k, v.do)[2].values()])
        graphs.append(graph)
    for i in range(3):
        v.x.copy_(C.normal((48, K), 1.0, 60 + i).to(T).cuda())
        for graph in graphs:
            graph.replay()
        o, k = v.forward(OG.SILU)
        want = [o, *v.backward(OG.SILU, k, v.do)[2].values()]
        torch.cuda.synchronize()
        for got in results:
            assert all(torch.equal(p, q) for p, q in zip(got, want)), i


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("m", [1, 16, 130])
def test_serving_in_8_bits(gpu_lib, m, act):
    lib, k, n = gpu_lib, 320, 700
    x, gain = C.normal((m, k), 1.0, 1).to(T).cuda(), C.normal((k,), 0.1, 2).add(1).to(T).cuda()
    wg = lib.quantize_int8(C.normal((2 * n, k), 1.5 / k ** 0.5, 3).float().cuda())
    wd = lib.quantize_int8(C.normal((k, n), 1 / n ** 0.5, 4).float().cuda())

    def run():
        x8, _ = lib.rmsnorm_int8(x, gain)
        p = lib.int8_linear_fwd_gated(wg, x8, act)
        p8 = lib.quantize_int8(p)
        return x8, p, p8, lib.int8_linear_fwd(wd, p8)

    value = lambda q: (q.codes[:, :q.k].cpu().double() * q.scale.cpu().double()[:, None])  # noqa: E731
    x8, p, p8, out = run()
    # the integer sums first, exact in float64: where one is zero, so is P
    sums = x8.codes.cpu().double() @ wg.codes.cpu().double().t().contiguous()
    y = (sums * torch.outer(x8.scale.cpu().double(), wg.scale.cpu().double())).numpy()
    g, u = y[:, :n], y[:, n:]
    p64 = OG.fwd(g, u, act)
    p_off = C.fwd_bound(g, u, act, T, 3 * C.F32 * np.abs(g), 3 * C.F32 * np.abs(u))
    C.check(p, p64, p_off, "P")
    # the rows of P round by half a step of their absmax / 127 more
    p8_off = torch.from_numpy(p_off) + p.cpu().double().abs().amax(1, keepdim=True) / 254 * 1.0001
    out64 = torch.from_numpy(p64) @ value(wd).t().contiguous()
    off = p8_off @ value(wd).abs().t().contiguous()
    C.check(out, out64.numpy(), ((out64.abs() + off) * (C.half_step(T) + 4 * C.F32) + off).numpy() + C.tiny(T), "out")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for i in range(3):
        x.copy_(C.normal((m, k), 1.0, 30 + i).to(T).cuda())
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert torch.equal(kept[1], want[1]) and torch.equal(kept[3], want[3]), i
