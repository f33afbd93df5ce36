"""GPU parity of the global gradient norm and clipping.

The norm's squares are summed in 64 bits: its relative error against the exact
one is below count 2^-53, so one float32 rounding apart, 2^-24 (and 2^-23 where
the two fall on both sides of a step). The factor is one float32 rounding of a
64-bit value (2^-24), the product one more, and the output's type one more:
relative tolerance 2^-23 + 2^-24 + half a step of the type."""
import math

import numpy as np
import pytest

from gpu_cases import say
from oracle import clip as OC

pytestmark = pytest.mark.gpu

HALF_STEP = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}

LISTS = {
    "one_element": [1],
    "small": [5, 0, 64, 1],
    "chunk_edges": [8191, 8192, 8193, 16383, 16384, 16385, 32768, 2047, 2048, 2049, 4097],
    "layer_rank8": [8 * 512, 512 * 8, 8 * 512, 1376 * 8, 8 * 1376],
    "many": [(37 * i) % 301 for i in range(500)],          # more than one launch's list, empties among them
    "exactly_one_slice": [100] * 240,
    "one_over_a_slice": [100] * 241,
    "two_slices_of_chunks": [2049, 5000, 1] * 160,
    "long": [3_000_001],
    "long_chunks": [4_194_305, 8191, 70_000, 8193],        # over 512 chunks of 8192: the longer chunks
}


def _grads(sizes, dtype, seed, std=1e-2):
    import torch

    rng = np.random.default_rng(seed)
    return [torch.from_numpy((rng.standard_normal(s) * std).astype(np.float32)).to(getattr(torch, dtype)).cuda()
            for s in sizes]


def _np(t):
    return t.detach().float().cpu().numpy()


def _near(got, want, dtype):
    tol = 2.0 ** -23 + 2.0 ** -24 + HALF_STEP[dtype]
    # below the type's normal range a step is absolute
    tiny = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -24}[dtype]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    g, w = got[ok].astype(np.float64), want[ok].astype(np.float64)
    assert np.all(np.abs(g - w) <= tol * np.abs(w) + tiny)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("name", sorted(LISTS))
def test_norm_and_clip(gpu_lib, name, dtype):
    import torch

    sizes = LISTS[name]
    say(f"[grad clip] {name} {dtype}")
    g = _grads(sizes, dtype, len(name))
    host = [_np(t) for t in g]
    total = OC.norm(host)
    n = gpu_lib.grad_norm(g)
    torch.cuda.synchronize()
    assert abs(float(n) - total) <= 2.0 ** -23 * total
    for max_norm in (0.5 * total, 2.0 * total, 0.0, math.inf):
        _, want = OC.clip(host, max_norm)
        out = torch.full((sum(sizes),), 3.0, dtype=g[0].dtype, device="cuda")
        n2 = gpu_lib.grad_clip(g, max_norm, out=out)
        torch.cuda.synchronize()
        assert float(n2) == float(n)
        assert all(np.array_equal(_np(t), h) for t, h in zip(g, host))  # the gradients are left as they were
        _near(_np(out), np.concatenate(want), dtype)
        mine = [t.clone() for t in g]
        kept = gpu_lib.GradList(mine)
        n3 = gpu_lib.grad_clip(kept, max_norm)
        torch.cuda.synchronize()
        assert float(n3) == float(n)
        assert np.array_equal(np.concatenate([_np(t) for t in mine]), _np(out))  # in place: the same bits


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_misaligned_tensors(gpu_lib, dtype):
    """Views at every element offset of a buffer, into an output at another
    offset; what lies around them keeps its values."""
    import torch

    t = getattr(torch, dtype)
    say(f"[grad clip] misaligned {dtype}")
    buf = torch.from_numpy(np.random.default_rng(1).standard_normal(60000).astype(np.float32)).to(t).cuda()
    before = buf.clone()
    cuts = [(1, 1001), (1005, 5003), (6010, 29991), (36005, 17)]
    g = [buf[a:a + s] for a, s in cuts]
    host = [_np(v) for v in g]
    total, want = OC.clip(host, 0.1)
    for shift in (0, 1, 3):
        hold = torch.full((sum(s for _, s in cuts) + 16,), 3.0, dtype=t, device="cuda")
        out = hold[shift:shift + sum(s for _, s in cuts)]
        n = gpu_lib.grad_clip(g, 0.1, out=out)
        torch.cuda.synchronize()
        assert abs(float(n) - total) <= 2.0 ** -23 * total
        _near(_np(out), np.concatenate(want), dtype)
        assert (hold[:shift] == 3).all() and (hold[shift + out.numel():] == 3).all()
    gpu_lib.grad_clip(g, 0.1)
    torch.cuda.synchronize()
    _near(np.concatenate([_np(v) for v in g]), np.concatenate(want), dtype)
    mask = torch.ones(60000, dtype=torch.bool, device="cuda")
    for a, s in cuts:
        mask[a:a + s] = False
    assert torch.equal(buf[mask], before[mask])


def test_not_finite(gpu_lib):
    import torch

    say("[grad clip] NaN and infinities")
    for bad, want_norm in ((float("nan"), math.nan), (float("inf"), math.inf), (float("-inf"), math.inf)):
        g = _grads([1000, 30], "float32", 2)
        g[1][7] = bad
        host = [_np(t) for t in g]
        total, want = OC.clip(host, 1.0)
        n = gpu_lib.grad_clip(g, 1.0)
        torch.cuda.synchronize()
        assert (math.isnan(float(n)) and math.isnan(total)) or float(n) == total == want_norm
        _near(np.concatenate([_np(t) for t in g]), np.concatenate(want), "float32")
    g = _grads([50], "float32", 3)
    g[0][3] = float("nan")
    keep = g[0].clone()
    gpu_lib.grad_clip(g, math.inf)  # nothing is scaled
    torch.cuda.synchronize()
    assert torch.equal(g[0].view(torch.int32), keep.view(torch.int32))


@pytest.mark.parametrize("scale", [1e30, 1e-30])
def test_squares_past_float32(gpu_lib, scale):
    import torch

    g = [torch.full((100,), scale, device="cuda")]
    n = gpu_lib.grad_norm(g)
    torch.cuda.synchronize()
    want = OC.norm([_np(g[0])])
    assert abs(float(n) - want) <= 2.0 ** -23 * want


def test_empty_lists(gpu_lib):
    import torch

    assert float(gpu_lib.grad_norm([])) == 0.0
    assert float(gpu_lib.grad_clip([], 1.0)) == 0.0
    none = torch.empty(0, device="cuda")
    assert float(gpu_lib.grad_clip([none, none], 1.0)) == 0.0
    assert float(gpu_lib.grad_clip([none], 1.0, out=torch.empty(0, device="cuda"))) == 0.0


def test_list_refusals_on_device(gpu_lib):
    """The same memory twice in place, an output over a gradient, and a length
    that changed since the list was made, are refused before any launch."""
    import torch

    g = _grads([100, 50], "float32", 4)
    keep = [t.clone() for t in g]
    with pytest.raises(gpu_lib.QloraError):
        gpu_lib.grad_clip([g[0], g[1], g[0]], 1e-3)
    with pytest.raises(gpu_lib.QloraError):
        gpu_lib.grad_clip([g[0][:60], g[0][59:]], 1e-3)
    big = torch.zeros(300, device="cuda")
    with pytest.raises(gpu_lib.QloraError):
        gpu_lib.grad_clip([big[100:150]], 1e-3, out=big[140:190])
    with pytest.raises(gpu_lib.QloraError):
        gpu_lib.grad_clip(g, float("nan"))
    with pytest.raises(gpu_lib.QloraError):
        gpu_lib.grad_clip(g, -1.0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(g, keep))
    # twice in the norm, and neighbours that touch, are fine
    two = gpu_lib.grad_norm([g[0], g[0]])
    gpu_lib.grad_clip([big[:100], big[100:]], 1.0)
    torch.cuda.synchronize()
    want = OC.norm([_np(g[0])] * 2)
    assert abs(float(two) - want) <= 2.0 ** -23 * want
    lst = gpu_lib.GradList(g)
    g[1].resize_(10)
    with pytest.raises(ValueError, match="changed its length"):
        gpu_lib.grad_norm(lst)


def test_backward_then_clip_in_one_graph(gpu_lib):
    """A layer's backward and the clipping of its dA and dB, captured once;
    every replay on new inputs equals the eager calls."""
    import torch

    from gpu_cases import layer_inputs

    n, k, m, r = 256, 320, 40, 8
    w, x, a, b, dy = layer_inputs(n, k, m, r, "clip_graph")
    q = gpu_lib.quantize(torch.from_numpy(w).cuda())
    x, a, b, dy = x.cuda(), a.cuda(), b.cuda(), dy.cuda()

    def step():
        _, da, db = gpu_lib.linear_bwd(q, x, dy, a, b, 16.0)
        return gpu_lib.grad_clip([da, db], 0.25), da, db

    say("[grad clip] backward and clip in a graph")
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(3):
        dy.copy_(torch.from_numpy(np.random.default_rng(i).standard_normal((m, n)).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, v) for p, v in zip(got, want))
        after = math.sqrt(sum(float(t.double().square().sum()) for t in got[1:]))
        assert float(got[0]) > 0.25
        # the 1e-6 beside the norm, and the factor's and the products' roundings
        assert abs(after - 0.25) <= 0.25 * (1e-6 / float(got[0]) + 2.0 ** -22)
