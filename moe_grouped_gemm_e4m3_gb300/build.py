"""Builds libdg.so (the sm_103a kernels and the C ABI of include/dg.h) in-tree with nvcc.

The translation units are compiled in parallel (one per GEMM form plus the API layer) and linked
into ``moe_grouped_gemm_e4m3_gb300/libdg.so``. ``_dgbind.so``, the binding's short path, is compiled beside it with the
host compiler against the installed torch's headers; if that fails, a message is printed and the binding
works without it. Rebuilds only when a source or header is newer than the library, and ``_dgbind.so`` also when torch or
Python is no longer the version it was compiled for. Usage: ``python -m moe_grouped_gemm_e4m3_gb300.build [--force]``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdg.so")
BIND = os.path.join(PKG, "_dgbind.so")
BIND_SRC = os.path.join(CSRC, "dg_bind.cpp")
BIND_KEY = os.path.join(BUILD_DIR, "dgbind.key")   # what the last compilation of _dgbind.so, good or not, was for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC,
              "--expt-relaxed-constexpr", "-diag-suppress", "177"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdg")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec is not None else None


def _bind_key() -> str:
    """The installed torch and Python, without importing torch (and its CUDA libraries)."""
    try:
        with open(os.path.join(_torch_dir() or "", "version.py")) as f:
            found = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M)
    except OSError:
        found = None
    return f"torch {found.group(1) if found else None} {sys.implementation.cache_tag}"


def bind_tried() -> bool:
    """Whether _dgbind.so was compiled, or failed to, from this source for this torch and Python."""
    if not os.path.exists(BIND_KEY):
        return False
    with open(BIND_KEY) as f:
        same = f.read() == _bind_key()
    return same and os.path.getmtime(BIND_KEY) >= max(os.path.getmtime(BIND_SRC), os.path.getmtime(os.path.abspath(__file__)))


def _bind_current() -> bool:
    return os.path.exists(BIND) and bind_tried()


def _start_bind():
    """The compilation of the binding's short path (None: no torch to compile against, or no compiler)."""
    torch_dir = _torch_dir()
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if torch_dir is None or not cxx:
        return None
    inc = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    lib = os.path.join(torch_dir, "lib")
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC"] + ["-I" + i for i in inc] + [BIND_SRC, "-o", tmp, "-L" + lib] + \
        ["-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl", "-Wl,-rpath," + lib]
    return tmp, _bind_key(), subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish_bind(started) -> None:
    if started is None:
        return
    tmp, key, proc = started
    out, _ = proc.communicate()
    if proc.returncode == 0:
        os.replace(tmp, BIND)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(BIND_KEY, "w") as f:
        f.write(key)
    if proc.returncode != 0:
        sys.stderr.write("the binding's short path did not compile (calls will check their arguments in Python):\n" +
                         out.decode(errors="replace")[-2000:])


def build(force: bool = False, verbose: bool = False) -> str:
    bind = None if not force and _bind_current() else _start_bind()
    try:
        return _build_lib(force, verbose)
    finally:
        _finish_bind(bind)


def _build_lib(force: bool, verbose: bool) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or verbose:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
