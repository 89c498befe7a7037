"""Kernels launched as programmatic dependents start while the kernel in front may still
be writing what they read.  A read-only load (__ldg, ld.global.nc, a const __restrict__
pointer) is defined only for memory that nothing writes during the kernel, so their
sources use none."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "token_indexed_sparse_staple_b200", "csrc")


def code_of(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["matmul_i8.cu", "norm.cu", "quant.cu", "rows.cuh"])
def test_no_read_only_loads(name):
    code = code_of(name)
    assert name.endswith("h") or "wait_prior_kernels();" in code
    assert not re.findall(r"__ldg|\.global\.(?:\w+\.)*nc\b|__restrict__", code)
