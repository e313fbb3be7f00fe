"""The few-token products' layouts, from the library's own header compiled by the host compiler."""
import ctypes
import functools
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_grouped_gemm_e4m3_gb300", "csrc")

SOURCE = """
#include "dg_few_plan.h"
using namespace dg;
extern "C" double few_choice_of(int T, int k, int E, int rows, int units, int four, int whole, int capped, long long* out) {
  const FewChoice c = few_choice(T, k, E, rows, units, four, whole, capped);
  out[0] = c.R, out[1] = c.plan.warps, out[2] = c.plan.ctas, out[3] = c.plan.stages, out[4] = (long long)c.plan.smem;
  return c.plan.cost;
}
extern "C" int few_stages_of(int T, int k, int E, int warps, int ctas, int R) {
  const int NT = few_tiles(T);
  return few_stages(warps, ctas, NT, R, routing_bytes(E, (T < 8 * NT ? T : 8 * NT) * k));
}
"""


@functools.cache
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, src, "-o", lib], check=True)
        loaded = ctypes.CDLL(lib)
    loaded.few_choice_of.restype = ctypes.c_double
    return loaded


def choice(T, k, E, rows, units, four=False, whole=True, capped=False):
    """(tiles of 16 rows a unit, warps, CTAs an SM, stages, shared memory, cost)"""
    out = (ctypes.c_longlong * 5)()
    cost = _lib().few_choice_of(T, k, E, rows, units, four, whole, capped, out)
    return (*out, cost)


def stages(T, k, E, warps, ctas, R):
    return _lib().few_stages_of(T, k, E, warps, ctas, R)


def layer(T, k, E, K, I, N, form, capped=False):
    """The layouts of the layer's two products."""
    four, unit = form == "mxfp4", 256 if form == "mxfp4" else 128
    most = min(T * k, E)
    return (choice(T, k, E, most * 2 * I, -(-K // unit), four, K % 256 == 0, capped),
            choice(T, k, E, N, -(-I // unit) * most, four, I % 256 == 0, capped))


def dense(M, N, K, capped=False):
    """The four-bit product's."""
    return choice(M, 0, 1, N, -(-K // 256), True, K % 256 == 0, capped)
