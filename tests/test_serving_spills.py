"""Build check, kernel by kernel: of the kernels of 8-bit floating-point serving only the cached attention's tiles hold scalars in
lanes of vector registers (up to 56: addresses, the table's and the masks' bounds, which their loop keeps); every other
kernel, those beside them in the same file too, holds none."""

import os
import re
import subprocess

import pytest

from bit_w4a4_quantized_quantize_amd import build
from tests.test_kernel_resources import HIPCC

# parts of the kernels' names in each source
KERNELS = {"fp8.hip": {"quant_fp8_kernel", "quant_weight_fp8_kernel", "gemm_fp8_kernel", "fp8_reduce_kernel", "gemm_fp8_few_kernel"},
           "cache.hip": {"append_kernel", "read_kernel"},
           "attention_cache.hip": {"attention_few_kernel", "attention_tile_kernel", "join_kernel"}}


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", sorted(KERNELS))
def test_scalars_of_each_kernel(src, tmp_path):
    cmd = [HIPCC, *build.COMMON_FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "--cuda-device-only", "-c",
           os.path.join(build.CSRC, src), "-o", str(tmp_path / "k.o"), "-Rpass-analysis=kernel-resource-usage"]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", out.stderr)
    spills = [int(v) for v in re.findall(r"SGPRs Spill: (\d+)", out.stderr)]
    assert names and len(names) == len(spills)
    seen = set()
    for name, n in zip(names, spills):
        kernel = max((k for k in KERNELS[src] if k in name), key=len)
        seen.add(kernel)
        assert n <= (56 if kernel == "attention_tile_kernel" else 0), (name, n)
    assert seen == KERNELS[src]
