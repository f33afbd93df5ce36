"""Memory of the backward from 8-bit rows without dX, and both least workspaces, on the GPU."""
import numpy as np
import pytest
import torch

import gated_cases as C
import test_gpu_linear_gated as L
import test_gpu_linear_x8 as X
from oracle import gated as OG

pytestmark = pytest.mark.gpu
T = torch.bfloat16


@pytest.mark.parametrize("n,k,parts", [(1024, 4096, 1), (4608, 1088, 1), (1024, 1088, 2)])
def test_no_room_for_a_weight_that_is_not_restored(gpu_lib, n, k, parts):
    m, r = 300, 16
    args = X.layer(gpu_lib, m, n, k, parts, r, T, 4)
    least = gpu_lib.x8_workspace_bytes(m, n, k, parts, r, restored=False)
    assert gpu_lib.x8_workspace_bytes(m, n, k, parts, r) >= least + 2 * n * k  # with dX it is restored
    want = X.call(gpu_lib, *args, parts)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    none, da, db = X.call(gpu_lib, *args, parts, need_dx=False)
    took = torch.cuda.max_memory_allocated() - before
    assert none is None and torch.equal(da, want[1]) and torch.equal(db, want[2])
    assert took <= least + da.nbytes + db.nbytes + 3 * 512, (took, least)
    ws = torch.full((least + 256,), 9, dtype=torch.uint8, device="cuda")
    _, da, db = X.call(gpu_lib, *args, parts, need_dx=False, ws=ws[:least])
    assert torch.equal(da, want[1]) and torch.equal(db, want[2]) and (ws[least:] == 9).all()


def test_a_block_in_its_least_workspace(gpu_lib):
    m, half, k, r = 70, 512, 320, 16
    w, x, a, b, alpha = L.layer(gpu_lib, m, half, k, r, T, 31)
    least = gpu_lib.gated_workspace_bytes(m, 2 * half, k, r, restored=False)
    ws = torch.full((least + 256,), 9, dtype=torch.uint8, device="cuda")
    g, u, _, dg, du, _ = L.expected(gpu_lib, w, x, a, b, alpha, T)
    p, y, _ = gpu_lib.linear_fwd_gated(w, x, a, b, alpha, ws=ws[:least])
    C.check(p, OG.fwd(g, u, OG.SILU), C.fwd_bound(g, u, OG.SILU, T, dg, du), "P")
    v, off = np.concatenate([g, u], 1), np.concatenate([dg, du], 1)
    C.check(y, v, np.abs(v) * C.half_step(T) * (1 + 2 ** -7) + off * 1.01 + C.tiny(T), "Y")
    assert (ws[least:] == 9).all()
