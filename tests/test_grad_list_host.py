"""A prepared gradient list refuses tensors that changed since it was made (no
GPU: every refusal here comes before the one of CPU tensors)."""
import pytest
import torch

from bit_nf4_quantized_18_amd import binding as B

CALLS = {"norm": lambda g: B.grad_norm(g), "clip": lambda g: B.grad_clip(g, 1.0),
         "clip_out": lambda g: B.grad_clip(g, 1.0, out=torch.zeros(30))}


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("at", [0, 1])
def test_replaced_data_is_refused(call, at):
    """A narrower type of the same length would be read, and in place written,
    past its end; one of the same width, and a strided view, give other values."""
    new = {0: lambda: torch.zeros(10), 1: lambda: torch.zeros(4, 5)}[at]
    wide = {0: lambda: torch.zeros(20)[::2], 1: lambda: torch.zeros(5, 4).t()}[at]
    for kind, data, err, match in (
            (torch.float32, new().bfloat16(), TypeError, f"gradient {at} has dtype torch.bfloat16"),
            (torch.float32, new().double(), TypeError, f"gradient {at} has dtype torch.float64"),
            (torch.bfloat16, new().half(), TypeError, f"gradient {at} has dtype torch.float16"),
            (torch.float32, wide(), ValueError, f"gradient {at} must be contiguous"),
            (torch.float32, torch.zeros(21), ValueError, "changed its length")):
        grads = [torch.zeros(10, dtype=kind), torch.zeros(4, 5, dtype=kind)]
        held = B.GradList(grads)
        grads[at].data = data
        with pytest.raises(err, match=match):
            CALLS[call](held)


def test_replaced_device_is_refused():
    """The list's GPU and the tensors' differ."""
    grads = [torch.zeros(10), torch.zeros(20)]
    held = B.GradList(grads)
    held.index = 0  # as a list made on GPU 0 has it
    for call in CALLS.values():
        with pytest.raises(ValueError, match="gradient 0 is on cpu, the list on GPU 0"):
            call(held)


def test_new_data_of_the_same_kind_is_taken():
    """The refusal that remains is the one of CPU tensors."""
    grads = [torch.zeros(10), torch.zeros(4, 5)]
    held = B.GradList(grads)
    grads[1].data = torch.ones(4, 5)
    assert list(held._pointers()) == [g.data_ptr() for g in grads]
    with pytest.raises(ValueError, match="on the GPU"):
        B.grad_norm(held)


def test_status_text_of_alignment():
    """The gradient calls refuse by element size, not by 16 bytes."""
    text = B.status_string(-3)
    assert "16 bytes" in text and "element size" in text
