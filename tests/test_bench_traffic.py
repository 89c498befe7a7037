"""The decode kernel's DRAM bytes come from a capture that holds for the sources it was
taken from: headers that the kernel includes hold what it needs, and what other kernels
alone need stands in headers of their own."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_the_decode_kernel_is_the_captured_one():
    c = bench.CAPTURED_TRAFFIC["k5k6_decode_fused"]
    assert bench.captured_traffic("k5k6_decode_fused") == (c["bytes"], c["profile"])
