"""What the layer operators' source may not hold."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "zero_sharded_optimizer_device_gb300", "csrc")
EARLY = ["zero_ops_device.cuh", "zero_linear.cu", "zero_rows.cu", "zero_dropout.cu", "zero_lnorm.cu"]


@pytest.mark.parametrize("name", EARLY)
def test_kernels_that_start_early_load_coherently(name):
    """These kernels start while the one before them on the stream still
    writes, perhaps the very layer buffer they read: a non-coherent load asks
    for memory that nobody writes while the kernel runs, and may be moved
    across the wait for the kernel before."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg|\bld\.global(\.\w+)*\.nc\b|\bld\.global\.nc\b|__restrict__|\bld_once\b", code)
