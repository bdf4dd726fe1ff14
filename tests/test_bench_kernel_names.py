"""bench.py's summaries of a profile know every kernel over lists of tensors."""
import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

with open(os.path.join(ROOT, "gram_newton_schulz_amd", "csrc", "gns_tensors.hip")) as f:
    KERNELS = sorted(set(re.findall(r"__global__[^;{]*?\b(\w+)\(ListView|__global__ void (\w+)\(int64_t", f.read())))
KERNELS = sorted(a or b for a, b in KERNELS)


def test_kernels_of_the_source():
    assert {"list_partials", "list_norm_once", "list_finish", "list_scale", "list_adamw"} <= set(KERNELS)


@pytest.mark.parametrize("kernel", KERNELS)
def test_kernel_has_its_row(kernel):
    name = f"void gns::(anonymous namespace)::{kernel}<false, true>(gns::ListView, unsigned long*)"
    assert bench.short_kernel(name) == kernel
    assert kernel in bench.HBM_KERNELS
