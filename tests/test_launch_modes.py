"""The early-start setting without a GPU: what it returns can be passed back."""
import os
import subprocess
import sys

import pytest

import moe_grouped_gemm_e4m3_gb300 as dg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("before", [None, False, True])
@pytest.mark.parametrize("inside", [None, False, True])
def test_the_previous_setting_can_be_restored(before, inside):
    first = dg.dg_set_pdl(before)
    try:
        assert dg.dg_get_pdl() is before
        prev = dg.dg_set_pdl(inside)
        assert prev is before and dg.dg_get_pdl() is inside
        assert dg.dg_set_pdl(prev) is inside
        assert dg.dg_get_pdl() is before
    finally:
        dg.dg_set_pdl(first)


@pytest.mark.parametrize("env,want", [(None, None), ("0", False), ("1", True)])
def test_the_environment_sets_the_initial_setting(env, want):
    e = {k: v for k, v in os.environ.items() if k != "DG_PDL"}
    e["PYTHONPATH"] = ROOT
    if env is not None:
        e["DG_PDL"] = env
    code = "import moe_grouped_gemm_e4m3_gb300 as dg; print(dg.dg_get_pdl(), dg.load().dg_get_pdl())"
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=e, check=True, stdout=subprocess.PIPE, text=True).stdout.split()
    assert out == [str(want), {None: "-1", False: "0", True: "1"}[want]]
