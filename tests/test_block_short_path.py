"""The compiled short path of the binding for the operators around the experts' products, without a GPU: it declines what it cannot take,
raises what the Python checks raise, and makes its calls without the interpreter's lock."""
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

import moe_grouped_gemm_e4m3_gb300 as dg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = """
import torch
import moe_grouped_gemm_e4m3_gb300 as dg
from torch._subclasses.fake_tensor import FakeTensorMode
with FakeTensorMode():
    t = lambda dt, *s: torch.zeros(s, dtype=getattr(torch, dt), device="cuda")
    x, v, u, a, sa, w1, s1, w2, s2, y = (t("bfloat16", 256, 256), t("float32", 256), t("float32", 256), t("uint8", 4, 256), t("float32", 2, 4),
        t("uint8", 3, 256, 256), t("float32", 3, 2, 2), t("uint8", 3, 256, 128), t("float32", 3, 2, 1), t("bfloat16", 4, 256))
    ids, w, l, b4, s4 = t("int32", 4, 2), t("float32", 4, 2), t("float32", 4, 3), t("uint8", 256, 128), t("uint8", 256, 8)
assert dg._bind() is not dg._NoBind
try:
    %s
except (RuntimeError, ValueError, TypeError) as e:
    print("raised", type(e).__name__)
"""
CALLS = {
    "norm": "dg.dg_residual_norm(x, v, Y=x)",
    "norm_backward": "dg.dg_residual_norm_backward(x, x, v, u, dX=x, dW=u)",
    "route": "dg.dg_route_topk(l, ids, w)",
    "route_backward": "dg.dg_route_topk_backward(w, l, ids, l)",
    "moe": "dg.dg_fp8_moe_swiglu(a, sa, w1, s1, w2, s2, ids, w, y)",
    "mxfp4": "dg.dg_fp8_mxfp4_gemm_nt(a, sa, b4, s4, y)",
}


@pytest.mark.parametrize("what", CALLS)
def test_tensors_without_memory_raise(what):
    assert dg._bind() is not dg._NoBind, "the short path is not built"
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""), CUDA_VISIBLE_DEVICES="")
    p = subprocess.run([sys.executable, "-c", FAKE % CALLS[what]], cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert p.returncode == 0 and "raised" in p.stdout, p.stdout[-2000:]


def _shell(dtype, *shape):
    """A tensor that says it is on the GPU and has no memory (nothing reads it here)."""
    import torch

    class Shell(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError(f"{func} on a tensor without memory")

    return torch.Tensor._make_wrapper_subclass(Shell, shape, dtype=getattr(torch, dtype), device="cuda")


def test_calls_release_the_lock_and_other_places_are_declined(tmp_path):
    """Against a library whose entry points return whether the caller holds the interpreter's lock. Without a driver the short path
    cannot know the current device: it declines, and nothing is called."""
    from moe_grouped_gemm_e4m3_gb300 import build
    src, lib, bind = tmp_path / "stand_in.c", tmp_path / "libstandin.so", tmp_path / "_dgbind.so"
    src.write_text("int PyGILState_Check(void);\n" + "".join(f"int {n}() {{ return PyGILState_Check(); }}\n" for n in dg.EXPORTED_SYMBOLS))
    subprocess.run([os.environ.get("CC") or "gcc", "-std=c11", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    dg._bind()
    shutil.copy(build.BIND, bind)
    loader = importlib.machinery.ExtensionFileLoader("_dgbind", str(bind))
    m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_dgbind", str(bind), loader=loader))
    loader.exec_module(m)
    assert m.load(str(lib))
    import torch
    x, v = _shell("bfloat16", 256, 256), _shell("float32", 256)
    got = [m.norm(0, x, None, None, None, None, v, 1e-6, None, x, None, None, None, None, 0),
           m.norm_backward(x, None, x, None, v, None, None, None, v, None, x, None, None, None, None, None, None, 0),
           m.route(0, _shell("float32", 4, 8), None, _shell("int32", 4, 2), _shell("float32", 4, 2), 0, True, 1.0, 0),
           m.mxfp4(0, _shell("uint8", 4, 256), _shell("float32", 2, 4), _shell("uint8", 64, 128), _shell("uint8", 64, 8), _shell("bfloat16", 4, 64), 0)]
    want = 0 if torch.cuda.is_available() else None
    assert got == [want] * 4, got
    # not a bool, not a float, too many dimensions, another size: declined
    assert m.route(0, _shell("float32", 4, 8), None, _shell("int32", 4, 2), _shell("float32", 4, 2), 0, 1, 1.0, 0) is None
    assert m.norm(0, x, None, None, None, None, _shell("float32", 255), 1e-6, None, x, None, None, None, None, 0) is None
    assert m.norm(0, _shell("bfloat16", 2, 2, 2), None, None, None, None, v, 1e-6, None, x, None, None, None, None, 0) is None
    assert m.moe(0, *[x] * 9, None, 0) is None and m.mxfp4(0, x) is None
