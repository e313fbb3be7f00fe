"""The compiled short path of the binding, without a GPU: it declines what it cannot take, and never ends the process.

Torch's accessors throw C++ exceptions for tensors without plain sizes or memory. Each such call runs in a
process of its own, which has to end with the Python exception that the checks in Python raise.
"""
import os
import subprocess
import sys

import pytest

import moe_grouped_gemm_e4m3_gb300 as dg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NESTED = """
import warnings; warnings.simplefilter("ignore")
x = torch.nested.nested_tensor([torch.zeros(3, 4), torch.zeros(2, 4)])
call = lambda: dg.dg_dropout(x, x, None, 0.0)
"""
FAKE = """
from torch._subclasses.fake_tensor import FakeTensorMode
u8, bf, f32, i32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
with FakeTensorMode():
    t = lambda dt, *s: torch.zeros(s, dtype=dt, device="cuda")
    a, b, sa, sb = t(u8, 256, 256), t(u8, 256, 256), t(f32, 2, 256), t(f32, 2, 2)
    d, h, bg, sbg, idx, off, dk = t(bf, 256, 256), t(bf, 256, 128), t(u8, 2, 256, 256), t(f32, 2, 2, 2), t(i32, 256), t(i32, 3), t(bf, 2, 256, 256)
call = lambda: %s
"""
CALLS = {
    "nested": NESTED,
    "dense": FAKE % "dg.dg_fp8_gemm_nt(a, sa, b, sb, d)",
    "layout": FAKE % "dg.dg_fp8_gemm_tn(a, sa, b, sb, d, 256, 256, 256)",
    "contiguous": FAKE % "dg.dg_fp8_grouped_contiguous(a, sa, bg, sbg, idx, d)",
    "contiguous_nn": FAKE % "dg.dg_fp8_grouped_contiguous_nn(a, sa, bg, sbg, idx, d)",
    "k_grouped": FAKE % "dg.dg_fp8_k_grouped_gemm_tn_contiguous(a, sa, b, sb, off, dk)",
    "gated": FAKE % "dg.dg_fp8_gemm_nt_swiglu(a, sa, b, sb, h)",
    "backward": FAKE % "dg.dg_swiglu_backward_fp8(h, d, a, sa)",
    "cast": FAKE % "dg.dg_cast_fp8(d, Xr=a, sR=sa)",
    "dropout": FAKE % "dg.dg_dropout(d, d, None, 0.0)",
}


def _run(body):
    code = "import torch\nimport moe_grouped_gemm_e4m3_gb300 as dg\n" + body
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""), CUDA_VISIBLE_DEVICES="")
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


@pytest.mark.parametrize("what", CALLS)
def test_tensors_without_memory_raise(what):
    assert dg._bind() is not dg._NoBind, "the short path is not built"
    p = _run(CALLS[what] + """
assert dg._bind() is not dg._NoBind
try:
    call()
except (RuntimeError, ValueError, TypeError) as e:
    print("raised", type(e).__name__)
""")
    assert p.returncode == 0 and "raised" in p.stdout, p.stdout[-2000:]
