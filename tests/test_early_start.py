"""Kernels that start before the launch ahead of them has ended (griddepcontrol) may not use read-only loads: those are for data
that nobody writes while the kernel lives, and the launch ahead still writes what such a kernel reads behind its wait."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_grouped_gemm_e4m3_gb300", "csrc")
FILES = ["dg_few.cu", "dg_norm.cu", "dg_route.cu", "dg_kernel.cuh", "dg_kernel_bs.cuh", "dg_gated_few.cu", "dg_cast.cu", "dg_dropout.cu"]
PARTS = ["dg_gated.cuh", "dg_philox.cuh", "dg_ptx.cuh", "dg_vec.cuh", "dg_scale.cuh"]   # of such kernels


def _code(name):
    """The source without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_every_such_source_is_here():
    found = {os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu*")) if "griddep_wait()" in open(f).read()}
    assert found - {"dg_ptx.cuh"} == set(FILES)


@pytest.mark.parametrize("name", FILES + PARTS)
def test_no_read_only_loads(name):
    code = _code(name)
    assert re.findall(r"__ldg\w*\(|ld\.global\.nc|ld\.global\.\S*\.nc|__restrict__", code) == []
