"""Build check: the kernels between the linears compile for gfx950 without scratch memory or register spills."""

import os

import pytest

from tests.test_kernel_resources import HIPCC
from tests.test_kernel_resources import test_no_scratch_no_spills as _check


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", ["int8.hip", "norm.hip", "rope.hip", "attention.hip"])
def test_no_scratch_no_spills_between_the_linears(src, tmp_path):
    _check(src, tmp_path)
