"""Build check: scalar registers that the kernels between the linears spill (into lanes of vector registers; the checks
of vector spills and scratch memory do not see them). None, but for attention's, where up to 39 loop constants are read back
by one instruction each while the next tiles are requested: 4 to 13 of about 1000 instructions for two tiles."""

import os
import re
import subprocess

import pytest

from bit_w4a4_quantized_quantize_amd import build
from tests.test_kernel_resources import HIPCC


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src,most", [("int8.hip", 0), ("norm.hip", 0), ("rope.hip", 0), ("attention.hip", 40)])
def test_scalar_spills(src, most, tmp_path):
    cmd = [HIPCC, *build.COMMON_FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "--cuda-device-only", "-c",
           os.path.join(build.CSRC, src), "-o", str(tmp_path / "k.o"), "-Rpass-analysis=kernel-resource-usage"]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", out.stderr)
    spills = [int(v) for v in re.findall(r"SGPRs Spill: (\d+)", out.stderr)]
    assert names and len(names) == len(spills)
    assert max(spills) <= most, dict(zip(names, spills))
