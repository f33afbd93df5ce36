"""dG = dP U act'(G) where U act' alone leaves float32 (act' > 1 next to U at the end of its range) and the result does not."""
import numpy as np
import pytest
import torch

import gated_cases as C
from oracle import gated as OG

pytestmark = pytest.mark.gpu

GATES = [1.5, 2.4, 3.0, 5.0, 1.2, 0.8, -0.5, 40.0]  # act' up to 1.0998 (SiLU) and 1.129 (GELU); below 1; 1
DPS = [0.1, -0.25, 1e-3, 0.9, 1e-30]


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_ups_at_the_end_of_their_range(gpu_lib, kind, act, rows):
    t = C.TYPES[kind]
    if rows:  # gates are codes of 0.1 (24 codes: 2.4), ups the largest codes of a scale
        gate = torch.tensor([round(10 * g) if abs(g) < 12 else 120 for g in GATES], dtype=torch.int8)
        up = torch.tensor([127, -127, 126, 120, 119, -118, 100, 127], dtype=torch.int8)
        scale = torch.tensor([0.1, 2.67e36])  # 127 of it: 3.39e38
        g, u = C.f64(gate.float() * scale[0]), C.f64(up.float() * scale[1])
        n, m = len(GATES), len(DPS)
        codes = torch.zeros(2 * m, 64, dtype=torch.int8)
        codes[0::2, :n], codes[1::2, :n] = gate, up
        y = gpu_lib.PackedInt8(2 * m, n, codes.cuda(), scale.repeat(m).cuda())
    else:
        gate = torch.tensor(GATES).to(t)
        up = torch.tensor([3.2e38, -3.38e38, 3.3e38, 1.8e38, 1.6e38, -3.2e38, 3.38e38, 3.38e38]).to(t)
        g, u = C.f64(gate), C.f64(up)
        n, m = len(GATES), len(DPS)
        y = torch.cat([gate, up])[None].expand(m, 2 * n).contiguous().cuda()
    dp = torch.tensor(DPS).to(t)[:, None].expand(m, n).contiguous()
    dg = C.f64(gpu_lib.gated_bwd(y, dp.cuda(), act))[:, :n]
    want = OG.bwd(g[None], u[None], C.f64(dp), act)[0]
    past = np.abs(want) > 3.41e38  # float32 ends at 3.403e38, bf16 at 3.39e38
    assert (np.abs(want[~past]) < 3.38e38).all() and not past.all(axis=0).any()
    # act' of these gates is 0.2 or more, its error (float32) below 2^-18 of 1, and in 16 bits below 2^-16
    rel = C.half_step(t) * 4 + (2.0 ** -13 if kind == "bf16" else 2.0 ** -15)
    assert np.array_equal(dg[past], np.sign(want[past]) * np.inf) and np.isfinite(dg[~past]).all(), dg
    assert (np.abs(dg - want)[~past] <= rel * np.abs(want)[~past]).all(), (dg, want)


def test_a_result_past_the_range_is_infinite(gpu_lib):
    y = torch.tensor([[2.4, 2.4, 3.3e38, -3.3e38]]).cuda()
    dg = gpu_lib.gated_bwd(y, torch.ones(1, 2).cuda(), OG.SILU)[0, :2]
    assert dg[0] == float("inf") and dg[1] == -float("inf")
