"""Kernels that split their registers among their warps: a split that does not add up to what the kernel was built with waits
for ever on the GPU, in a place that no bounded wait covers, so the host has to ask before a launch."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNITS = [p for p in sorted(glob.glob(os.path.join(ROOT, "gguf_block_dequant_gb300", "csrc", "*.cu"))) if "setmaxnreg" in open(p).read()]


def test_there_are_such_units():
    assert {os.path.basename(p) for p in UNITS} >= {"qg_attn_tc.cu", "qg_delta_chunk.cu"}


@pytest.mark.parametrize("path", UNITS, ids=os.path.basename)
def test_the_host_asks_for_the_registers(path):
    """The answer decides about the launch, and the shares of three warpgroups stay within what the launch gives them."""
    text = open(path).read()
    asked = re.search(r"(\w+) = qg::split_fits\([^;]*, (\w+)\);", text)
    assert asked, "no check before the launch"
    assert re.search(rf"if \([^;{{]*!?\b{asked[1]}\b", text)
    assert re.search(rf"constexpr int [^;]*\b{asked[2]} = \d+", text)
    assert re.search(rf"static_assert\([^;]*<= [^;]*{asked[2]}", text)
