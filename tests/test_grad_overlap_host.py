"""The gradient calls refuse a norm or a workspace that overlaps the gradients,
the output or each other (no GPU: fake addresses). The norm is written while
other workgroups still read partial sums and gradients, the workspace while the
gradients are read."""
import ctypes

import pytest

from bit_nf4_quantized_18_amd import binding as B

F32, BF16 = B.QLORA_F32, B.QLORA_BF16
SIZES = [100, 0, 5000]
AT = [1 << 20, 0, 2 << 20]
NORM, WS, OUT = 3 << 20, 4 << 20, 5 << 20


def _calls(t):
    lib = B.load()
    ptr, num = (ctypes.c_void_p * 3)(*AT), (ctypes.c_int64 * 3)(*SIZES)
    need = lib.qlora_grad_workspace_bytes(num, 3)

    def norm(norm=NORM, ws=WS, nbytes=need, p=ptr):
        return lib.qlora_grad_norm(p, num, 3, t, norm, ws, nbytes, None)

    def clip(norm=NORM, ws=WS, nbytes=need, o=None, p=ptr):
        return lib.qlora_grad_clip(p, num, 3, t, 1.0, o, norm, ws, nbytes, None)

    return norm, clip, need


@pytest.mark.parametrize("t,size", [(F32, 4), (BF16, 2)])
def test_norm_and_workspace_over_a_gradient(t, size):
    norm, clip, need = _calls(t)
    for f in (norm, clip, lambda **kw: clip(o=OUT, **kw)):
        for at, n in ((AT[0], 100), (AT[2], 5000)):
            assert f(norm=at) == -4 and f(norm=at + (n * size - 4) // 4 * 4) == -4
            assert f(ws=at) == -4 and f(ws=at + (n * size - 1) // 16 * 16) == -4 and f(ws=at - (need - 1) // 16 * 16) == -4


@pytest.mark.parametrize("t", [F32, BF16])
def test_norm_in_the_workspace(t):
    norm, clip, need = _calls(t)
    for f in (norm, clip, lambda **kw: clip(o=OUT, **kw)):
        for at in (WS, WS + 4, WS + need - 4):
            assert f(norm=at) == -4


@pytest.mark.parametrize("t,size", [(F32, 4), (BF16, 2)])
def test_output_over_norm_and_workspace(t, size):
    _, clip, need = _calls(t)
    total = sum(SIZES) * size
    for at in (NORM, NORM - total + 4):
        assert clip(o=at) == -4
    for at in (WS, WS + need - size, WS - total + size):
        assert clip(o=at) == -4


@pytest.mark.parametrize("t", [F32, BF16])
def test_an_empty_tensor_meets_nothing(t):
    """Its address may lie in the norm, the workspace or another tensor: the
    call is taken and ends at the launch, for which there is no GPU."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses are no memory of a GPU")
    norm, clip, _ = _calls(t)
    for inside in (NORM, WS + 8, AT[2] + 16, AT[0], OUT + 8):
        p = (ctypes.c_void_p * 3)(AT[0], inside, AT[2])
        for f in (norm, clip, lambda **kw: clip(o=OUT, **kw)):
            assert f(p=p) == -6
