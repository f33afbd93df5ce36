"""The rule that chooses whether a product restores its weight once, compiled for the host."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("rule") / "dense_rule")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I" + os.path.join(ROOT, "bit_nf4_quantized_18_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "dense_rule_emul.cpp"), "-o", exe], check=True)

    def ask(cases):
        text = "".join("%d %d %d\n" % c for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return ask


def test_choices_follow_the_measured_sides(rule):
    # (tokens, outputs, contraction) -> whether restoring once was measured to be faster, where the sides are over 5% apart
    measured = {(64, 22016, 4096): 0, (2048, 22016, 4096): 1, (4096, 22016, 4096): 1, (64, 44032, 8192): 0,
                (2048, 44032, 8192): 1, (64, 2560, 5120): 1, (333, 2560, 5120): 1, (4096, 2560, 5120): 1,
                (64, 5120, 1088): 1, (333, 5120, 1088): 1, (2048, 5120, 1088): 1, (4096, 5120, 1088): 1,
                (64, 4096, 22016): 1, (256, 4096, 22016): 1, (1024, 4096, 22016): 1, (4096, 4096, 22016): 1,
                (64, 11008, 4096): 1, (256, 11008, 4096): 1, (1024, 11008, 4096): 1, (4096, 11008, 4096): 1,
                (64, 22016, 8192): 0, (256, 22016, 8192): 0, (1024, 22016, 8192): 0, (2048, 4096, 22016): 0}
    got = rule(list(measured))
    assert [g for _, g, _ in got] == list(measured.values())
    assert all(f for f, _, _ in got)


def test_bounds(rule):
    (fits, _, _), (long_fits, long_pays, _), most, more = rule([(17, 512, 65536), (17, 512, 65600), ((1 << 22) - 1, 512, 64),
                                                          (1 << 22, 512, 64)])
    assert fits == 1 and long_fits == 0 and long_pays == 0
    assert most[0] == 1 and more[:2] == (0, 0)  # a launch of 2^32 threads


def test_tokens_by_sixteen_where_that_was_measured_to_be_faster(rule):
    cases = {(16, 512, 64): 1, (16, 44032, 8192): 1, (17, 1024, 1024): 0, (32, 5120, 1088): 0, (32, 11264, 2048): 1,
             (17, 10240, 2560): 1, (32, 16384, 4096): 1, (32, 22016, 4096): 1, (33, 22016, 4096): 0, (32, 28672, 4096): 1,
             (32, 27648, 5120): 1, (17, 44032, 8192): 1, (33, 28672, 4096): 0}
    assert [d for _, _, d in rule(list(cases))] == list(cases.values())
