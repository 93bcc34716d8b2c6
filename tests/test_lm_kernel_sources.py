"""The register and scratch budget (test_kernel_resources.py) is held by every HIP source of the 8-bit
operators and the mixture-of-experts layer too: they are among the sources it compiles."""
import os
import re

from linear_algebra_sgemm_amd import build, resource_usage


def test_every_kernel_source_is_compiled():
    listed = {os.path.basename(s) for s in resource_usage.hip_sources()}
    assert {"quantize_kernels.hip", "fp8_kernels.hip", "fp8_tile_kernels.hip",
            "moe_kernels.hip"} <= listed
    for name in os.listdir(build.CSRC):
        with open(os.path.join(build.CSRC, name)) as f:
            if name.endswith(".hip") and re.search(r"__global__", f.read()):
                assert name in listed, name
