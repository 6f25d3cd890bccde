"""Build check: the kernels of 8-bit floating-point serving compile for gfx950 without scratch memory or spills of vector
registers. Scalar registers that do not fit are held in lanes of vector registers, without a memory access: the cached
attention's tiles, whose loop keeps the tensors' addresses, the table's and the masks' bounds there, hold up to 56 so,
and nothing else any."""

import os
import re
import subprocess

import pytest

from bit_w4a4_quantized_quantize_amd import build
from tests.test_kernel_resources import HIPCC


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src,scalars", [("fp8.hip", 0), ("cache.hip", 0), ("attention_cache.hip", 56), ("rope.hip", 0)])
def test_no_scratch_no_spills(src, scalars, tmp_path):
    cmd = [HIPCC, *build.COMMON_FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "--cuda-device-only", "-c",
           os.path.join(build.CSRC, src), "-o", str(tmp_path / "k.o"), "-Rpass-analysis=kernel-resource-usage"]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", out.stderr)
    for what, most in (("ScratchSize \\[bytes/lane\\]", 0), ("VGPRs Spill", 0), ("SGPRs Spill", scalars)):
        found = [int(v) for v in re.findall(what + r": (\d+)", out.stderr)]
        assert names and len(found) == len(names)
        assert max(found) <= most, (what, dict(zip(names, found)))
