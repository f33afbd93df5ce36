"""The 8-bit product at contractions that end at every place of a tile's ring:
behind at least one whole turn of it and without one. Each such end is code of
its own over counted waits. Which tile a size takes is asserted, without a GPU,
in test_int8_tiles_host.py; results are bit-equal to the oracle's."""
import pytest

from gpu_cases import say
from oracle import int8 as OI

pytestmark = pytest.mark.gpu

# m, n, k -> tile, units of 128 codes (of one group) behind the last whole turn
TAILS = [(1610, 5037, 317), (1480, 5405, 448),      # 256 x 256, 3 and 4 without a turn
         (1741, 4611, 700), (2316, 3500, 960),      # 256 x 256, 1 and 3
         (519, 3686, 704),                          # 128 x 128, 2
         (197, 4212, 690),                          # 64 x 128, 2
         (2072, 67, 320), (2104, 65, 704),          # 64 x 64, 3 without a turn, 2
         (2099, 65, 1664), (17, 68, 1570)]          # 32 x 64, 16 x 64: 3 in two groups


@pytest.mark.parametrize("size", TAILS, ids=lambda s: "x".join(map(str, s)))
def test_linear_every_tail(gpu_lib, size):
    import numpy as np
    import torch

    m, n, k = size
    say(f"[int8 linear] tails m={m} n={n} k={k}")
    rng = np.random.default_rng(m + n + k)
    ld = -(-k // 64) * 64

    def rows(count):
        codes = np.zeros((count, ld), np.int8)
        codes[:, :k] = rng.integers(-127, 128, (count, k))
        return codes, (10.0 ** rng.uniform(-3, -1, count)).astype(np.float32)

    (w, sw), (x, sx) = rows(n), rows(m)
    want = torch.from_numpy(OI.linear(w, sw, x, sx))
    packed = lambda c, s: gpu_lib.PackedInt8(len(s), k, torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda())  # noqa: E731
    qw, qx = packed(w, sw), packed(x, sx)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        y = torch.full((m, n), 7.0, dtype=dtype, device="cuda")
        gpu_lib.int8_linear_fwd(qw, qx, dtype, out=y)
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), want.to(dtype))
