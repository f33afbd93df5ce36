"""The gated block in 8-bit integers against float64."""
import numpy as np
import pytest
import torch

import gated_cases as C
from oracle import gated as OG

pytestmark = pytest.mark.gpu


def rows(n, k, seed):
    rng = np.random.default_rng(seed)
    codes = np.zeros((n, -(-k // 64) * 64), dtype=np.int8)
    codes[:, :k] = rng.integers(-127, 128, (n, k))
    return torch.from_numpy(codes), torch.from_numpy(rng.uniform(0.5, 1.5, n).astype(np.float32))


def case(lib, m, n, k, seed, sx=1 / 1000, sw=1 / 1000):
    xc, xs = rows(m, k, seed)
    wc, ws = rows(2 * n, k, seed + 1)
    xs, ws = xs * sx, ws * sw / max(1.0, k ** 0.5 / 16)
    acc = xc.double() @ wc.double().t().contiguous()  # exact
    v = (acc * torch.outer(xs.double(), ws.double())).numpy()
    x = lib.PackedInt8(m, k, xc.cuda(), xs.cuda())
    w = lib.PackedInt8(2 * n, k, wc.cuda(), ws.cuda())
    return w, x, v[:, :n], v[:, n:]


# every tile, the streaming kernel, both sides of 16 tokens, ragged sizes, odd halves, short and long contractions
SIZES = [(1, 1, 64), (1, 7, 100), (16, 8, 64), (3, 129, 4100), (16, 4095, 128), (1, 11008, 512), (17, 24, 64), (40, 100, 1000),
         (130, 333, 320), (64, 4096, 256), (300, 1030, 700), (1000, 2051, 192), (513, 5504, 128), (260, 4300, 1088)]


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("kind", list(C.TYPES))
@pytest.mark.parametrize("m,n,k", SIZES)
def test_block(gpu_lib, m, n, k, kind, act):
    t = C.TYPES[kind]
    w, x, g, u = case(gpu_lib, m, n, k, m + n + k)
    p = gpu_lib.int8_linear_fwd_gated(w, x, act, t)
    assert p.dtype is t and p.shape == (m, n)
    # the sum's rounding to float32 and the two scales': three roundings
    bound = C.fwd_bound(g, u, act, t, 3 * C.F32 * np.abs(g), 3 * C.F32 * np.abs(u))
    C.check(p, OG.fwd(g, u, act), bound, "P")


def test_rows_do_not_depend_on_the_batch(gpu_lib):
    w, x, _, _ = case(gpu_lib, 300, 700, 256, 5)
    whole = gpu_lib.int8_linear_fwd_gated(w, x)
    for i in (0, 4, 252):
        one = gpu_lib.PackedInt8(4, x.k, x.codes[i:i + 4], x.scale[i:i + 4])
        assert torch.equal(gpu_lib.int8_linear_fwd_gated(w, one), whole[i:i + 4])


def test_agrees_with_the_two_calls(gpu_lib):
    w, x, _, _ = case(gpu_lib, 50, 300, 640, 8)
    y = gpu_lib.int8_linear_fwd(w, x, torch.float32)
    for act in C.ACTS:
        assert torch.equal(gpu_lib.int8_linear_fwd_gated(w, x, act, torch.float32), gpu_lib.gated_fwd(y, act))


def test_output_in_its_own_rows(gpu_lib):
    m, n = 21, 301
    w, x, _, _ = case(gpu_lib, m, n, 128, 2)
    room = torch.full((m * n + 100,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = room[: m * n].view(m, n)
    assert gpu_lib.int8_linear_fwd_gated(w, x, out=out) is out
    assert torch.equal(out, gpu_lib.int8_linear_fwd_gated(w, x)) and (room[m * n:] == 3.0).all()
    with pytest.raises(gpu_lib.QloraError):
        gpu_lib.int8_linear_fwd_gated(w, x, out=w.codes.view(torch.bfloat16).view(-1)[: m * n].view(m, n))


def test_values_that_are_not_finite(gpu_lib):
    w, x, _, _ = case(gpu_lib, 5, 40, 64, 3)
    x.scale[2] = float("nan")
    w.scale[7] = float("nan")  # a gate
    w.scale[40 + 9] = float("nan")  # an up
    p = gpu_lib.int8_linear_fwd_gated(w, x)
    bad = torch.isnan(p)
    assert bad[2].all() and bad[:, 7].all() and bad[:, 9].all()
    bad[2], bad[:, 7], bad[:, 9] = False, False, False
    assert not bad.any()


def test_no_tokens(gpu_lib):
    w, _, _, _ = case(gpu_lib, 1, 40, 64, 3)
    none = gpu_lib.PackedInt8(0, 64, torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    assert gpu_lib.int8_linear_fwd_gated(w, none).shape == (0, 40)
