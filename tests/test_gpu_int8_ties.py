"""Codes next to ties on the GPU, bit-equal to the oracle's: through the
quantizer and the norm, in rows of one wave, of a workgroup and of the two
passes, at magnitudes on both sides of the 64-bit path's."""
import pytest

import int8_ties
from gpu_cases import say
from oracle import int8 as OI

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [0, -24, 60, -120])
@pytest.mark.parametrize("cols", [8, 300, 4001, 30001])
def test_codes_next_to_ties(gpu_lib, cols, exponent):
    import numpy as np
    import torch

    say(f"[int8 ties] cols={cols} exponent={exponent}")
    v = int8_ties.rows(exponent)
    x = np.zeros((len(v), cols), np.float32)
    for at in range(0, cols - 7, 8):
        x[:, at:at + 8] = v
    x[:, cols - 7:] = v[:, 1:]  # an odd row's end
    x[:, 0] = v[:, 0]
    codes, scale = OI.quantize(x)
    q = gpu_lib.quantize_int8(torch.from_numpy(x).cuda())
    torch.cuda.synchronize()
    assert np.array_equal(q.codes.cpu().numpy()[:, :cols], codes)
    assert np.array_equal(q.scale.cpu().numpy().view(np.uint32), scale.view(np.uint32))
    # a gain of one leaves the values, so the norm's codes are the same
    gain = torch.ones(cols, device="cuda")
    n, _ = gpu_lib.rmsnorm_int8(torch.from_numpy(x).cuda(), gain, 0.0)
    torch.cuda.synchronize()
    assert np.array_equal(n.codes.cpu().numpy()[:, :cols], codes)
    codes_n, scale_n, _ = OI.rmsnorm(x, np.ones(cols, np.float32), 0.0)
    assert np.array_equal(codes_n, codes)
    got = n.scale.cpu().numpy().astype(np.float64)
    # the 64-bit sum's order, and one float32 rounding on each side
    assert np.all(np.abs(got - scale_n) <= 2.0 ** -23 * scale_n)


def test_subnormal_scales(gpu_lib):
    import numpy as np
    import torch

    say("[int8 ties] subnormal scales")
    steps = np.concatenate([np.arange(1, 700), 127 * np.arange(1, 300) + 63, 127 * np.arange(1, 300) + 64])
    x = np.zeros((len(steps), 16), np.float32)
    x[:, 5] = np.ldexp(steps.astype(np.float64), -149)
    x[::2] *= -1
    codes, scale = OI.quantize(x)
    q = gpu_lib.quantize_int8(torch.from_numpy(x).cuda())
    torch.cuda.synchronize()
    assert np.array_equal(q.codes.cpu().numpy()[:, :16], codes)
    assert np.array_equal(q.scale.cpu().numpy().view(np.uint32), scale.view(np.uint32))
