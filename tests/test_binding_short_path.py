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


@pytest.fixture(scope="module")
def against_a_stand_in(tmp_path_factory):
    """The short path loaded with a library whose entry points return whether the caller holds the interpreter's lock."""
    import importlib.machinery
    import importlib.util
    import shutil

    from moe_grouped_gemm_e4m3_gb300 import build
    d = tmp_path_factory.mktemp("stand_in")
    src, lib, bind = d / "stand_in.c", d / "libstandin.so", d / "_dgbind.so"
    src.write_text("int PyGILState_Check(void);\n" + "".join(f"int {n}() {{ return PyGILState_Check(); }}\n" for n in dg.EXPORTED_SYMBOLS))
    subprocess.run([os.environ.get("CC") or "gcc", "-std=c11", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    dg._bind()                                   # torch's libraries are loaded
    shutil.copy(build.BIND, bind)                # a file of its own: its entry points are not the binding's
    loader = importlib.machinery.ExtensionFileLoader("_dgbind", str(bind))
    mod = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_dgbind", str(bind), loader=loader))
    loader.exec_module(mod)
    assert mod.load(str(lib))
    return mod


def _shell(dtype, *shape):
    """A tensor that says it is on the GPU and has no memory (nothing reads it here)."""
    import torch

    class Shell(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError(f"{func} on a tensor without memory")

    return torch.Tensor._make_wrapper_subclass(Shell, shape, dtype=getattr(torch, dtype), device="cuda")


def test_the_interpreter_runs_on_during_a_call(against_a_stand_in):
    """A launch can wait for a full queue; other threads of Python must not wait with it."""
    u8, bf, f32, i32 = ((lambda *s, d=d: _shell(d, *s)) for d in ("uint8", "bfloat16", "float32", "int32"))
    a, sa, b, sb, d = u8(256, 256), f32(2, 256), u8(256, 256), f32(2, 2), bf(256, 256)
    bg, sbg, idx, h, dk = u8(2, 256, 256), f32(2, 2, 2), i32(256), bf(256, 128), bf(2, 256, 256)
    m = against_a_stand_in
    calls = [m.dense(0, a, sa, b, sb, d, 256, 256, 256, 0), m.contiguous(0, a, sa, bg, sbg, idx, d, 0),
             m.contiguous(4, a, sa, bg, sbg, idx, d, 0), m.k_grouped(0, a, sa, b, sb, i32(3), dk, 0),
             m.gated(0, a, sa, b, sb, None, h, None, None, 0.0, 0), m.gated(4, a, sa, bg, sbg, idx, h, None, None, 0.0, 0),
             m.backward(0, h, d, a, sa, None, None, None, None, None, None, 0.0, 0),
             m.cast(0, d, a, sa, None, None, None, None, None, None, 0), m.dropout(d, None, d, None, 0.0, 0)]
    assert calls == [0] * len(calls), calls      # (None: declined; 1: called with the lock held)


def test_another_torch_asks_for_another_short_path(tmp_path, monkeypatch):
    """The short path is compiled against torch's headers: an upgraded torch, whose files keep older dates, makes it stale."""
    import importlib.util
    import types

    from moe_grouped_gemm_e4m3_gb300 import build
    assert dg._bind() is not dg._NoBind and build._bind_current()
    (tmp_path / "version.py").write_text("__version__ = '99.0.0+cu999'\n")
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: types.SimpleNamespace(submodule_search_locations=[str(tmp_path)]))
    assert not build._bind_current()
