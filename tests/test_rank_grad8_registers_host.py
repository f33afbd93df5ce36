"""The kernel of dA and dB from 8-bit rows holds its loads ahead in registers (no GPU; compiles the file): a spilled load
has to arrive before it can be stored, so its step would wait for it. One address may be spilled."""
import os
import re
import subprocess

import pytest

from bit_nf4_quantized_18_amd import build as B


def test_no_load_ahead_is_spilled(tmp_path):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    src, out = os.path.join(B.CSRC, "rank_grad8.hip"), str(tmp_path / "rank_grad8.out")
    p = subprocess.run([B.HIPCC] + B.COMMON + B.SOURCES["rank_grad8.hip"] + ["--cuda-device-only", "-S", src, "-o", out],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    text = open(out).read()
    found = dict(re.findall(r"\.name: +(\S+)[\s\S]*?\.vgpr_spill_count: +(\d+)", text[text.index("amdhsa.kernels"):]))
    kernels = {k: int(v) for k, v in found.items() if "rank_grad8_kernel" in k}
    assert len(kernels) == 4 and max(kernels.values()) <= 4, kernels
    # a run of scratch accesses is a group of registers put aside; an address is two
    for run in re.findall(r"(?:^\s+scratch_(?:load|store)\S* .*\n)+", text, re.M):
        assert run.count("scratch_") <= 2, run
