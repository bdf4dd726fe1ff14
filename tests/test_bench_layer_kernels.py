"""bench.py's summaries of a profile know every kernel of the layers."""
import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

KERNELS = []
for source in ("gns_embedding.hip", "gns_mxfp4.hip"):
    with open(os.path.join(ROOT, "gram_newton_schulz_amd", "csrc", source)) as f:
        KERNELS += re.findall(r"__global__ void(?: __launch_bounds__\((?:\([^()]*\)|[^()])*\))?\s+(\w+)\(", f.read())


def test_kernels_of_the_sources():
    assert set(KERNELS) == set(bench.LAYER_KERNELS) and len(KERNELS) == len(bench.LAYER_KERNELS)


@pytest.mark.parametrize("kernel", KERNELS)
def test_kernel_has_its_row(kernel):
    name = f"void gns::(anonymous namespace)::{kernel}<gns::EBF16, (gns::Spread)1, true>(gns::Sums, float*)"
    assert bench.short_kernel(name) == kernel
    assert kernel in bench.HBM_KERNELS
