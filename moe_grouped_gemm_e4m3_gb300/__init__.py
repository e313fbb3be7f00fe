"""FP8 (E4M3) fine-grained-scaled GEMM for GB300 — thin Python binding of libdg (include/dg.h).

Argument marshalling only: every step of the GEMM runs in the sm_103a kernels of ``libdg.so``.
PyTorch supplies device memory and the current CUDA stream. There is no fallback: if the library
is missing or cannot load, every call raises.

The names mirror the C ABI:

* ``dg_fp8_gemm_nt(A, sA, B, sB, D)``                       dense D = A·Bᵀ
* ``dg_fp8_grouped_contiguous(A, sA, B, sB, m_indices, D)``  M-grouped, contiguous layout
* ``dg_fp8_grouped_masked(A, sA, B, sB, masked_m, D)``       M-grouped, masked layout
* ``*_f32`` variants store the FP32 accumulator instead of BF16 (same kernel and order).
* ``dg_fp8_gemm_{nn,tn,tt}(A, sA, B, sB, D, M=, N=, K=)``     dense D = A·Bᵀ with A stored [K,M] (t) and/or
  B stored [K,N] (second letter n); the scales keep dg_fp8_gemm_nt's layouts
* ``dg_fp8_k_grouped_gemm_tn_contiguous(A, sA, B, sB, k_offsets, D)``  groups along K: A [K,M], B [K,N],
  D [G,M,N]
* ``dg_fp8_grouped_masked_swiglu(A, sA, B, sB, masked_m, H)``  masked GEMM + SwiGLU: B [G, 2I, K], H [G, M_max, I]
* ``dg_fp8_gemm_nt_acc_f32(A, sA, B, sB, C, D)``             D = C + A·Bᵀ (FP32 C and D; C may be D)
* ``dg_fp8_gemm_nt_swiglu(A, sA, B, sB, H, GU=, rng=, p=)``   gated projection H = dropout(silu(gate)·up), dense;
  ``dg_fp8_grouped_contiguous_swiglu`` over contiguous groups; GU [rows, 2I] saves the pre-activations
* ``dg_swiglu_backward_fp8(dH, GU, dGUr, sR, dGUc, sC, Hb=, sHb=, ...)``  its backward pass up to the products, cast to E4M3
* ``dg_fp8_grouped_contiguous_nn(A, sA, B, sB, m_indices, D)``  contiguous layout with B stored [G, K, N]
* ``dg_cast_fp8(X, Xr=, sR=, Xc=, sC=, Xb=, sB=, sBt=, m_indices=)``  BF16 to E4M3 with 1x128, 128x1 and 128x128 scales
* ``dg_dropout(X, Y, rng, p, R=)``  Y = R + dropout(X) from a counter-based generator, BF16 or FP32
* ``*_ue8m0`` variants take power-of-two scales as packed UE8M0 int32 words (four K-groups per
  word, byte j = K-group 4q+j): sA int32 [ceil(ceil(K/128)/4), align4(rows)] (masked: leading G),
  sB int32 [G, ceil(N/128), ceil(ceil(K/128)/4)]. They run the block-scaled tensor-core kernel.

Tensor contract (all CUDA, contiguous): A uint8/float8_e4m3fn [rows, K] (masked: [G, M_max, K]);
B uint8/float8_e4m3fn [N, K] or [G, N, K]; sA float32 MN-major [ceil(K/128), align4(rows)]
(masked: [G, ceil(K/128), align4(M_max)]); sB float32 [G, ceil(N/128), ceil(K/128)]; D bfloat16
(or float32) [rows, N] (masked: [G, M_max, N]); m_indices / masked_m int32.
"""
from __future__ import annotations

import ctypes
import functools
import os

from . import build as _build_mod

__all__ = [
    "DGError", "load", "dg_fp8_gemm_nt", "dg_fp8_gemm_nt_f32", "dg_fp8_grouped_contiguous",
    "dg_fp8_grouped_contiguous_f32", "dg_fp8_grouped_masked", "dg_fp8_grouped_masked_f32", "dg_fp8_gemm_nt_noalloc",
    "dg_get_tma_aligned_size", "dg_get_mk_alignment_for_contiguous_layout", "dg_set_num_sms",
    "dg_get_num_sms", "dg_get_device_status", "dg_last_error_string", "dg_query_config",
    "dg_set_tail_splits", "dg_set_cluster_split", "dg_set_wait_limit_us", "dg_set_pair_b", "dg_set_pdl", "dg_get_pdl",
    "dg_transform_sf_into_ue8m0_a", "dg_transform_sf_into_ue8m0_b", "dg_transform_sf_a_into_mn_major",
    "dg_fp8_gemm_nt_ue8m0", "dg_fp8_gemm_nt_ue8m0_f32", "dg_fp8_grouped_contiguous_ue8m0",
    "dg_fp8_grouped_contiguous_ue8m0_f32", "dg_fp8_grouped_masked_ue8m0", "dg_fp8_grouped_masked_ue8m0_f32",
    "dg_query_config_ue8m0", "dg_fp8_gemm_nt_acc_f32", "dg_fp8_gemm_nt_ue8m0_acc_f32",
    "dg_fp8_grouped_masked_swiglu", "dg_fp8_grouped_masked_swiglu_f32", "dg_fp8_grouped_masked_swiglu_fp8",
    "dg_fp8_grouped_masked_swiglu_ue8m0",
    "dg_fp8_grouped_masked_swiglu_ue8m0_f32", "dg_fp8_gemm_nn", "dg_fp8_gemm_nn_f32",
    "dg_fp8_gemm_tn", "dg_fp8_gemm_tn_f32", "dg_fp8_gemm_tt", "dg_fp8_gemm_tt_f32",
    "dg_fp8_gemm_nn_ue8m0", "dg_fp8_gemm_nn_ue8m0_f32", "dg_fp8_gemm_tn_ue8m0", "dg_fp8_gemm_tn_ue8m0_f32", "dg_fp8_gemm_tt_ue8m0", "dg_fp8_gemm_tt_ue8m0_f32",
    "dg_fp8_k_grouped_gemm_tn_contiguous", "dg_fp8_k_grouped_gemm_tn_contiguous_f32",
    "dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0", "dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0_f32", "EXPORTED_SYMBOLS", "DG_OK", "DG_ERR_INVALID_ARG", "DG_ERR_ALIGNMENT", "DG_ERR_UNSUPPORTED",
    "DG_ERR_CUDA", "DG_ERR_DEVICE_STATUS", "DG_DEV_BAD_GROUP_INDEX", "DG_DEV_BAD_MASKED_M",
    "DG_DEV_TIMEOUT", "DG_DEV_BAD_SCALE",
    "dg_fp8_gemm_nt_swiglu", "dg_fp8_gemm_nt_swiglu_f32", "dg_fp8_gemm_nt_swiglu_ue8m0",
    "dg_fp8_gemm_nt_swiglu_ue8m0_f32", "dg_fp8_grouped_contiguous_swiglu",
    "dg_fp8_grouped_contiguous_swiglu_f32", "dg_fp8_grouped_contiguous_swiglu_ue8m0",
    "dg_fp8_grouped_contiguous_swiglu_ue8m0_f32", "dg_fp8_grouped_contiguous_nn",
    "dg_fp8_grouped_contiguous_nn_f32", "dg_fp8_grouped_contiguous_nn_ue8m0",
    "dg_fp8_grouped_contiguous_nn_ue8m0_f32", "dg_swiglu_backward_fp8", "dg_swiglu_backward_fp8_ue8m0",
    "dg_cast_fp8", "dg_cast_fp8_ue8m0", "dg_dropout",
]

DG_OK, DG_ERR_INVALID_ARG, DG_ERR_ALIGNMENT, DG_ERR_UNSUPPORTED, DG_ERR_CUDA, DG_ERR_DEVICE_STATUS = range(6)
DG_DEV_BAD_GROUP_INDEX, DG_DEV_BAD_MASKED_M, DG_DEV_TIMEOUT, DG_DEV_BAD_SCALE = 0x1, 0x2, 0x4, 0x8

# Every symbol include/dg.h declares (checked against the built library by the CPU tests).
EXPORTED_SYMBOLS = (
    "dg_fp8_gemm_nt", "dg_fp8_gemm_nt_f32", "dg_fp8_grouped_contiguous", "dg_fp8_grouped_contiguous_f32",
    "dg_fp8_grouped_masked", "dg_fp8_grouped_masked_f32", "dg_get_tma_aligned_size",
    "dg_get_mk_alignment_for_contiguous_layout", "dg_set_num_sms", "dg_get_num_sms", "dg_get_device_status",
    "dg_last_error_string", "dg_query_config", "dg_fp8_gemm_nt_noalloc", "dg_set_tail_splits",
    "dg_set_cluster_split", "dg_set_wait_limit_us", "dg_set_pair_b", "dg_set_pdl", "dg_get_pdl",
    "dg_transform_sf_into_ue8m0_a", "dg_transform_sf_into_ue8m0_b", "dg_transform_sf_a_into_mn_major",
    "dg_fp8_gemm_nt_ue8m0", "dg_fp8_gemm_nt_ue8m0_f32", "dg_fp8_grouped_contiguous_ue8m0",
    "dg_fp8_grouped_contiguous_ue8m0_f32", "dg_fp8_grouped_masked_ue8m0", "dg_fp8_grouped_masked_ue8m0_f32",
    "dg_query_config_ue8m0", "dg_fp8_gemm_nt_acc_f32", "dg_fp8_gemm_nt_ue8m0_acc_f32",
    "dg_fp8_grouped_masked_swiglu", "dg_fp8_grouped_masked_swiglu_f32", "dg_fp8_grouped_masked_swiglu_fp8",
    "dg_fp8_grouped_masked_swiglu_ue8m0",
    "dg_fp8_grouped_masked_swiglu_ue8m0_f32", "dg_fp8_gemm_nn", "dg_fp8_gemm_nn_f32",
    "dg_fp8_gemm_tn", "dg_fp8_gemm_tn_f32", "dg_fp8_gemm_tt", "dg_fp8_gemm_tt_f32",
    "dg_fp8_gemm_nn_ue8m0", "dg_fp8_gemm_nn_ue8m0_f32", "dg_fp8_gemm_tn_ue8m0", "dg_fp8_gemm_tn_ue8m0_f32", "dg_fp8_gemm_tt_ue8m0", "dg_fp8_gemm_tt_ue8m0_f32",
    "dg_fp8_k_grouped_gemm_tn_contiguous", "dg_fp8_k_grouped_gemm_tn_contiguous_f32",
    "dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0", "dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0_f32",
    "dg_fp8_gemm_nt_swiglu", "dg_fp8_gemm_nt_swiglu_f32", "dg_fp8_gemm_nt_swiglu_ue8m0",
    "dg_fp8_gemm_nt_swiglu_ue8m0_f32", "dg_fp8_grouped_contiguous_swiglu",
    "dg_fp8_grouped_contiguous_swiglu_f32", "dg_fp8_grouped_contiguous_swiglu_ue8m0",
    "dg_fp8_grouped_contiguous_swiglu_ue8m0_f32", "dg_fp8_grouped_contiguous_nn",
    "dg_fp8_grouped_contiguous_nn_f32", "dg_fp8_grouped_contiguous_nn_ue8m0",
    "dg_fp8_grouped_contiguous_nn_ue8m0_f32", "dg_swiglu_backward_fp8", "dg_swiglu_backward_fp8_ue8m0",
    "dg_cast_fp8", "dg_cast_fp8_ue8m0", "dg_dropout_bf16", "dg_dropout_f32",
)


class DGError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libdg status {status}: {msg}")
        self.status = status


_lib = None


def load(build_if_missing: bool = True):
    """Loads libdg.so (building it first if it is missing or stale and nvcc is available)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build_mod.LIB
    if build_if_missing and not _build_mod.up_to_date():
        _build_mod.build()
    if not os.path.exists(path):
        raise DGError(DG_ERR_UNSUPPORTED, f"libdg.so not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, i32 = ctypes.c_void_p, ctypes.c_int
    for name in ("dg_fp8_gemm_nt", "dg_fp8_gemm_nt_f32", "dg_fp8_gemm_nt_noalloc", "dg_fp8_gemm_nt_ue8m0",
                 "dg_fp8_gemm_nt_ue8m0_f32", "dg_fp8_gemm_nn", "dg_fp8_gemm_nn_f32", "dg_fp8_gemm_tn",
                 "dg_fp8_gemm_tn_f32", "dg_fp8_gemm_tt", "dg_fp8_gemm_tt_f32", "dg_fp8_gemm_nn_ue8m0", "dg_fp8_gemm_nn_ue8m0_f32", "dg_fp8_gemm_tn_ue8m0", "dg_fp8_gemm_tn_ue8m0_f32", "dg_fp8_gemm_tt_ue8m0", "dg_fp8_gemm_tt_ue8m0_f32"):
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, [P, P, P, P, P, i32, i32, i32, P]
    for name in ("dg_fp8_grouped_contiguous", "dg_fp8_grouped_contiguous_f32", "dg_fp8_grouped_contiguous_ue8m0",
                 "dg_fp8_grouped_contiguous_ue8m0_f32"):
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, [P, P, P, P, P, P, i32, i32, i32, i32, P]
    for name in ("dg_fp8_grouped_masked", "dg_fp8_grouped_masked_f32", "dg_fp8_grouped_masked_ue8m0",
                 "dg_fp8_grouped_masked_ue8m0_f32", "dg_fp8_grouped_masked_swiglu",
                 "dg_fp8_grouped_masked_swiglu_f32", "dg_fp8_grouped_masked_swiglu_ue8m0",
                 "dg_fp8_grouped_masked_swiglu_ue8m0_f32"):
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, [P, P, P, P, P, P, i32, i32, i32, i32, P]
    lib.dg_fp8_grouped_masked_swiglu_fp8.restype = i32
    lib.dg_fp8_grouped_masked_swiglu_fp8.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, P]
    lib.dg_get_tma_aligned_size.restype, lib.dg_get_tma_aligned_size.argtypes = i32, [i32, i32]
    lib.dg_get_mk_alignment_for_contiguous_layout.restype = i32
    lib.dg_get_mk_alignment_for_contiguous_layout.argtypes = []
    lib.dg_set_num_sms.restype, lib.dg_set_num_sms.argtypes = None, [i32]
    lib.dg_get_num_sms.restype, lib.dg_get_num_sms.argtypes = i32, []
    lib.dg_set_tail_splits.restype, lib.dg_set_tail_splits.argtypes = i32, [i32]
    lib.dg_set_cluster_split.restype, lib.dg_set_cluster_split.argtypes = i32, [i32]
    lib.dg_set_pair_b.restype, lib.dg_set_pair_b.argtypes = i32, [i32]
    lib.dg_set_pdl.restype, lib.dg_set_pdl.argtypes = i32, [i32]
    lib.dg_get_pdl.restype, lib.dg_get_pdl.argtypes = i32, []
    for name in ("dg_transform_sf_into_ue8m0_a", "dg_transform_sf_into_ue8m0_b", "dg_transform_sf_a_into_mn_major"):
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, [P, P, i32, i32, i32, P]
    lib.dg_set_wait_limit_us.restype, lib.dg_set_wait_limit_us.argtypes = ctypes.c_longlong, [ctypes.c_longlong]
    lib.dg_get_device_status.restype, lib.dg_get_device_status.argtypes = i32, [ctypes.POINTER(i32), P]
    lib.dg_last_error_string.restype, lib.dg_last_error_string.argtypes = ctypes.c_char_p, []
    for name in ("dg_fp8_gemm_nt_acc_f32", "dg_fp8_gemm_nt_ue8m0_acc_f32"):
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, [P, P, P, P, P, P, i32, i32, i32, P]
    for name in ("dg_fp8_k_grouped_gemm_tn_contiguous", "dg_fp8_k_grouped_gemm_tn_contiguous_f32",
                 "dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0", "dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0_f32"):
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, [P, P, P, P, P, P, i32, i32, i32, i32, P]
    f64 = ctypes.c_double
    for ue in ("", "_ue8m0"):
        for f32 in ("", "_f32"):
            f = getattr(lib, f"dg_fp8_gemm_nt_swiglu{ue}{f32}")
            f.restype, f.argtypes = i32, [P, P, P, P, P, P, P, f64, i32, i32, i32, P]
            f = getattr(lib, f"dg_fp8_grouped_contiguous_swiglu{ue}{f32}")
            f.restype, f.argtypes = i32, [P, P, P, P, P, P, P, P, f64, i32, i32, i32, i32, P]
            f = getattr(lib, f"dg_fp8_grouped_contiguous_nn{ue}{f32}")
            f.restype, f.argtypes = i32, [P, P, P, P, P, P, i32, i32, i32, i32, P]
        f = getattr(lib, f"dg_swiglu_backward_fp8{ue}")
        f.restype, f.argtypes = i32, [P, P, P, P, f64, P, P, P, P, P, P, i32, i32, P]
        f = getattr(lib, f"dg_cast_fp8{ue}")
        f.restype, f.argtypes = i32, [P, P, P, P, P, P, P, P, P, i32, i32, i32, P]
    for name in ("dg_dropout_bf16", "dg_dropout_f32"):
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, [P, P, P, P, f64, ctypes.c_longlong, P]
    for name in ("dg_query_config", "dg_query_config_ue8m0"):
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, [i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
    _lib = lib
    return lib


def _check(status: int):
    if status != DG_OK:
        raise DGError(status, load().dg_last_error_string().decode(errors="replace"))


class _NoBind:
    """Stands in for the short path where it is not built: every call goes through the checks below."""
    gated = dense = contiguous = k_grouped = backward = cast = dropout = staticmethod(lambda *a: None)


@functools.cache
def _bind():
    """The compiled short path (csrc/dg_bind.cpp): checks the arguments of a call and makes it, or returns None where
    something is not as it should be; the checks below then say what."""
    import importlib.machinery
    import importlib.util

    import torch
    load()
    if not _build_mod.bind_tried():   # torch or Python changed since; without a compiler the calls are checked in Python
        try:
            _build_mod.build()
        except (RuntimeError, OSError):
            pass
    try:
        loader = importlib.machinery.ExtensionFileLoader("_dgbind", _build_mod.BIND)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_dgbind", _build_mod.BIND, loader=loader))
        loader.exec_module(mod)
    except (ImportError, OSError):
        return _NoBind
    same = mod.version() == torch.__version__.split("+")[0]   # (a process that outlived an upgrade on disk, or no compiler to follow it)
    return mod if same and mod.load(_build_mod.LIB) else _NoBind


# The variants of the entry points as the short path numbers them: bit 0 FP32 output, bit 1 packed UE8M0 scales.
@functools.cache
def _variant(name):
    return (1 if name.endswith("_f32") else 0) + (2 if "_ue8m0" in name else 0)


def _raw(stream):
    """A stream as the short path takes it: None (the current one) or its number."""
    return None if stream is None else int(getattr(stream, "cuda_stream", stream))


# The helpers below run on every call, so each has a short path for well-formed arguments (a few attribute
# reads, about 0.3 us a tensor) and leaves the words of an error to a second look.

def _stream(stream):
    if stream is None:
        c = _torch()._C
        return c._cuda_getCurrentRawStream(c._cuda_getDevice())   # torch.cuda.current_stream(), 0.2 us instead of 2.9
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


@functools.cache
def _torch():
    import torch
    torch.cuda.init()
    return torch


def _ptr(t, name, dtypes):
    try:
        if t.dtype in dtypes and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except (AttributeError, TypeError):
        pass
    if not isinstance(t, _tensor()):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    raise ValueError(f"{name} must be contiguous")


@functools.cache
def _tensor():
    import torch
    return torch.Tensor


def _shape(t, name):
    if not isinstance(t, _tensor()):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.shape


def _size(v, name):
    """An extent as the C entry points take it (ctypes would pass a larger one on modulo 2^32)."""
    if v > 0x7FFFFFFF:
        raise ValueError(f"{name} is {v}; the calls take extents below 2^31")
    return v


def _sizes(t, name):
    """The shape of a tensor whose extents go to a C entry point."""
    s = _shape(t, name)
    for v in s:
        if v > 0x7FFFFFFF:
            _size(v, f"an extent of {name}")
    return s


def _expect(t, name, shape):
    """Raises ValueError unless tensor `t` has exactly `shape` (checked before any pointer is taken,
    so that a mis-shaped call never reaches a kernel, whose TMA boxes would read out of bounds)."""
    got = _shape(t, name)
    if got != shape:
        raise ValueError(f"{name} has shape {list(got)}, expected {list(shape)}")


def _pointers(*tensors):
    """The pointers of (tensor, name, dtypes, shape) arguments, checked in one pass where all is well. Otherwise
    every shape is looked at before any pointer is taken, and the first thing wrong is named. The name of an
    optional argument ends in "?": None is a null pointer there."""
    ptrs = []
    try:
        for t, name, dtypes, shape in tensors:
            if t is None and name[-1] == "?":
                ptrs.append(None)
            elif t.dtype in dtypes and t.shape == shape and t.is_cuda and t.is_contiguous():
                ptrs.append(t.data_ptr())
            else:
                break
        else:
            return ptrs
    except (AttributeError, TypeError):
        pass
    given = [(t, name.rstrip("?"), dtypes, shape) for t, name, dtypes, shape in tensors if t is not None or name[-1] != "?"]
    for t, name, _, shape in given:
        _expect(t, name, shape)
    for t, name, dtypes, _ in given:
        _ptr(t, name, dtypes)
    raise AssertionError("unreachable: an argument was refused without a reason")


def _cdiv(a, b):
    return -(-a // b)


def _align4(x):
    return -(-x // 4) * 4


def _scale_k(name, K):
    """Scale entries along K: one per 128-deep K-block (FP32 scales), or one int32 word per four
    K-blocks (packed UE8M0)."""
    nkb = _cdiv(K, 128)
    return _cdiv(nkb, 4) if "_ue8m0" in name else nkb


@functools.cache
def _fp8_types():
    import torch
    return (torch.uint8, torch.float8_e4m3fn)


@functools.cache
def _f32():
    import torch
    return (torch.float32,)


@functools.cache
def _scale_types(name):
    import torch
    return (torch.int32,) if "_ue8m0" in name else (torch.float32,)


@functools.cache
def _d_types(f32: bool):
    import torch
    return (torch.float32,) if f32 else (torch.bfloat16, torch.int16, torch.uint16)


_NT = ("dg_fp8_gemm_nt", "dg_fp8_gemm_nt_f32", "dg_fp8_gemm_nt_ue8m0", "dg_fp8_gemm_nt_ue8m0_f32")


def _dense_shapes(name, A, B):
    """(M, N, K) of a dense call: A [M, K], B [N, K] (or [1, N, K])."""
    a, b = _sizes(A, "A"), _sizes(B, "B")
    if len(a) != 2:
        raise ValueError(f"A must be [M, K], got {list(a)}")
    if not (len(b) == 2 or (len(b) == 3 and b[0] == 1)):
        raise ValueError(f"B must be [N, K] (or [1, N, K]), got {list(b)}")
    M, K = a
    N = b[-2]
    if b[-1] != K:
        raise ValueError(f"B has K = {b[-1]}, A has K = {K}")
    return M, N, K


def _check_scales_2d(name, sA, sB, M, N, K):
    nks = _scale_k(name, K)
    _expect(sA, "sA", (nks, _align4(M)))
    sb = _sizes(sB, "sB")
    want = (_cdiv(N, 128), nks)
    if sb != want and sb != (1,) + want:
        raise ValueError(f"sB has shape {list(sb)}, expected {list(want)}")


def _dense(name, f32, A, sA, B, sB, D, stream):
    if name in _NT and getattr(A, "ndim", 0) == 2 and getattr(B, "ndim", 0) == 2:
        (M, K), N = A.shape, B.shape[0]
        status = _bind().dense(_variant(name), A, sA, B, sB, D, M, N, K, _raw(stream))
        if status is not None:
            _check(status)
            return D
    M, N, K = _dense_shapes(name, A, B)
    _check_scales_2d(name, sA, sB, M, N, K)
    q, st = _fp8_types(), _scale_types(name)
    ptrs = _pointers((A, "A", q, A.shape), (sA, "sA", st, sA.shape), (B, "B", q, B.shape), (sB, "sB", st, sB.shape),
                     (D, "D", _d_types(f32), (M, N)))
    _check(getattr(load(), name)(*ptrs, M, N, K, _stream(stream)))
    return D


def dg_fp8_gemm_nt(A, sA, B, sB, D, stream=None):
    """D[M,N] (bfloat16) = A[M,K]·B[N,K]ᵀ with fine-grained scales."""
    return _dense("dg_fp8_gemm_nt", False, A, sA, B, sB, D, stream)


def dg_fp8_gemm_nt_f32(A, sA, B, sB, D, stream=None):
    """As dg_fp8_gemm_nt, storing the FP32 accumulator."""
    return _dense("dg_fp8_gemm_nt_f32", True, A, sA, B, sB, D, stream)


def dg_fp8_gemm_nt_noalloc(A, sA, B, sB, D, stream=None):
    """As dg_fp8_gemm_nt, without any allocation: for callers that cannot let the library call
    cudaMalloc (a framework whose caching allocator owns device memory, a serving loop that must not
    block on cudaMalloc's synchronisation). Split-K scratch comes from a fixed 20 MiB array inside
    libdg shared by all calls on a device, so calls that overlap on the GPU race; a shape that needs
    more scratch raises DGError(DG_ERR_UNSUPPORTED). The first call on a device looks up the array's
    address; make it before any stream capture."""
    return _dense("dg_fp8_gemm_nt_noalloc", False, A, sA, B, sB, D, stream)


def _contig(name, f32, A, sA, B, sB, m_indices, D, stream):
    status = _bind().contiguous(_variant(name), A, sA, B, sB, m_indices, D, _raw(stream))
    if status is not None:
        _check(status)
        return D
    a, b = _sizes(A, "A"), _sizes(B, "B")
    if len(a) != 2 or len(b) != 3:
        raise ValueError(f"contiguous layout: A must be [M_total, K] and B [G, N, K], got {list(a)} and {list(b)}")
    M, K = a
    G, N = b[0], b[1]
    if b[2] != K:
        raise ValueError(f"B has K = {b[2]}, A has K = {K}")
    nks = _scale_k(name, K)
    _expect(sA, "sA", (nks, _align4(M)))
    _expect(sB, "sB", (G, _cdiv(N, 128), nks))
    _expect(m_indices, "m_indices", (M,))
    _expect(D, "D", (M, N))
    lib = load()
    _check(getattr(lib, name)(_ptr(A, "A", _fp8_types()), _ptr(sA, "sA", _scale_types(name)), _ptr(B, "B", _fp8_types()),
                              _ptr(sB, "sB", _scale_types(name)), _ptr(m_indices, "m_indices", _i32()),
                              _ptr(D, "D", _d_types(f32)), M, N, K, G, _stream(stream)))
    return D


def dg_fp8_grouped_contiguous(A, sA, B, sB, m_indices, D, stream=None):
    """Contiguous-layout grouped GEMM: row m of D uses expert m_indices[m] (-1: padding, untouched)."""
    return _contig("dg_fp8_grouped_contiguous", False, A, sA, B, sB, m_indices, D, stream)


def dg_fp8_grouped_contiguous_f32(A, sA, B, sB, m_indices, D, stream=None):
    return _contig("dg_fp8_grouped_contiguous_f32", True, A, sA, B, sB, m_indices, D, stream)


def _masked(name, f32, A, sA, B, sB, masked_m, D, stream):
    a, b = _sizes(A, "A"), _sizes(B, "B")
    if len(a) != 3 or len(b) != 3:
        raise ValueError(f"masked layout: A must be [G, M_max, K] and B [G, N, K], got {list(a)} and {list(b)}")
    G, M_max, K = a
    N = b[1]
    if b[0] != G or b[2] != K:
        raise ValueError(f"B has shape {list(b)}, expected [{G}, N, {K}]")
    nks = _scale_k(name, K)
    _expect(sA, "sA", (G, nks, _align4(M_max)))
    _expect(sB, "sB", (G, _cdiv(N, 128), nks))
    _expect(masked_m, "masked_m", (G,))
    # the fused SwiGLU writes H = silu(gate)·up, half as wide as B's 2I rows
    _expect(D, "H" if "swiglu" in name else "D", (G, M_max, N // 2 if "swiglu" in name else N))
    lib = load()
    _check(getattr(lib, name)(_ptr(A, "A", _fp8_types()), _ptr(sA, "sA", _scale_types(name)), _ptr(B, "B", _fp8_types()),
                              _ptr(sB, "sB", _scale_types(name)), _ptr(masked_m, "masked_m", _i32()),
                              _ptr(D, "D", _d_types(f32)), G, M_max, N, K, _stream(stream)))
    return D


def dg_fp8_grouped_masked(A, sA, B, sB, masked_m, D, stream=None):
    """Masked-layout grouped GEMM: rows m < masked_m[g] of group g are computed, the rest untouched."""
    return _masked("dg_fp8_grouped_masked", False, A, sA, B, sB, masked_m, D, stream)


def dg_fp8_grouped_masked_f32(A, sA, B, sB, masked_m, D, stream=None):
    return _masked("dg_fp8_grouped_masked_f32", True, A, sA, B, sB, masked_m, D, stream)


def _dense_acc(name, A, sA, B, sB, C, D, stream):
    M, N, K = _dense_shapes(name, A, B)
    _check_scales_2d(name, sA, sB, M, N, K)
    _expect(C, "C", (M, N))
    _expect(D, "D", (M, N))
    lib = load()
    _check(getattr(lib, name)(_ptr(A, "A", _fp8_types()), _ptr(sA, "sA", _scale_types(name)),
                              _ptr(B, "B", _fp8_types()), _ptr(sB, "sB", _scale_types(name)), _ptr(C, "C", _f32()),
                              _ptr(D, "D", _f32()), M, N, K, _stream(stream)))
    return D


def dg_fp8_gemm_nt_acc_f32(A, sA, B, sB, C, D, stream=None):
    """D (float32) = C + A·Bᵀ; C (float32 [M,N]) may be D itself."""
    return _dense_acc("dg_fp8_gemm_nt_acc_f32", A, sA, B, sB, C, D, stream)


def dg_fp8_gemm_nt_ue8m0_acc_f32(A, sA, B, sB, C, D, stream=None):
    """As dg_fp8_gemm_nt_acc_f32 with packed UE8M0 scales."""
    return _dense_acc("dg_fp8_gemm_nt_ue8m0_acc_f32", A, sA, B, sB, C, D, stream)


# The layouts' names: the first letter says how A is stored (n: [M, K], t: [K, M]), the second how
# B is stored (t: [N, K], n: [K, N]).
_LAYOUT_VARIANTS = {"nn": 4, "tn": 8, "tt": 12}
_LAYOUTS = {"nn": (False, True), "tn": (True, True), "tt": (True, False)}


def _dense_layout(name, f32, A, sA, B, sB, D, M, N, K, stream):
    status = _bind().dense(_variant(name) + _LAYOUT_VARIANTS[name[12:14]], A, sA, B, sB, D, M, N, K, _raw(stream))
    if status is not None:
        _check(status)
        return D
    a_t, b_n = _LAYOUTS[name[len("dg_fp8_gemm_"):len("dg_fp8_gemm_") + 2]]
    M, N, K = (_size(int(v), n) for v, n in ((M, "M"), (N, "N"), (K, "K")))
    nks, q, st = _scale_k(name, K), _fp8_types(), _scale_types(name)
    ptrs = _pointers((A, "A", q, (K, M) if a_t else (M, K)), (sA, "sA", st, (nks, _align4(M))),
                     (B, "B", q, (K, N) if b_n else (N, K)), (sB, "sB", st, (_cdiv(N, 128), nks)),
                     (D, "D", _d_types(f32), (M, N)))
    _check(getattr(load(), name)(*ptrs, M, N, K, _stream(stream)))
    return D


def dg_fp8_gemm_nn(A, sA, B, sB, D, M, N, K, stream=None):
    """D[M,N] = A·Bᵀ with A stored [M,K] and B stored [K,N] (N contiguous)."""
    return _dense_layout("dg_fp8_gemm_nn", False, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_nn_f32(A, sA, B, sB, D, M, N, K, stream=None):
    return _dense_layout("dg_fp8_gemm_nn_f32", True, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_tn(A, sA, B, sB, D, M, N, K, stream=None):
    """D[M,N] = A·Bᵀ with A stored [K,M] and B stored [K,N] (both M/N contiguous)."""
    return _dense_layout("dg_fp8_gemm_tn", False, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_tn_f32(A, sA, B, sB, D, M, N, K, stream=None):
    return _dense_layout("dg_fp8_gemm_tn_f32", True, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_tt(A, sA, B, sB, D, M, N, K, stream=None):
    """D[M,N] = A·Bᵀ with A stored [K,M] and B stored [N,K]."""
    return _dense_layout("dg_fp8_gemm_tt", False, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_tt_f32(A, sA, B, sB, D, M, N, K, stream=None):
    return _dense_layout("dg_fp8_gemm_tt_f32", True, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_nn_ue8m0(A, sA, B, sB, D, M, N, K, stream=None):
    """dg_fp8_gemm_nn with packed UE8M0 scales (sA [ceil(nkb/4), align4(M)], sB [ceil(N/128), ceil(nkb/4)] int32)."""
    return _dense_layout("dg_fp8_gemm_nn_ue8m0", False, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_nn_ue8m0_f32(A, sA, B, sB, D, M, N, K, stream=None):
    return _dense_layout("dg_fp8_gemm_nn_ue8m0_f32", True, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_tn_ue8m0(A, sA, B, sB, D, M, N, K, stream=None):
    """dg_fp8_gemm_tn with packed UE8M0 scales."""
    return _dense_layout("dg_fp8_gemm_tn_ue8m0", False, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_tn_ue8m0_f32(A, sA, B, sB, D, M, N, K, stream=None):
    return _dense_layout("dg_fp8_gemm_tn_ue8m0_f32", True, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_tt_ue8m0(A, sA, B, sB, D, M, N, K, stream=None):
    """dg_fp8_gemm_tt with packed UE8M0 scales."""
    return _dense_layout("dg_fp8_gemm_tt_ue8m0", False, A, sA, B, sB, D, M, N, K, stream)


def dg_fp8_gemm_tt_ue8m0_f32(A, sA, B, sB, D, M, N, K, stream=None):
    return _dense_layout("dg_fp8_gemm_tt_ue8m0_f32", True, A, sA, B, sB, D, M, N, K, stream)


def _k_grouped(name, f32, A, sA, B, sB, k_offsets, D, stream):
    status = _bind().k_grouped(_variant(name), A, sA, B, sB, k_offsets, D, _raw(stream))
    if status is not None:
        _check(status)
        return D
    a, b, o = _sizes(A, "A"), _sizes(B, "B"), _sizes(k_offsets, "k_offsets")
    if len(a) != 2 or len(b) != 2 or len(o) != 1 or o[0] < 1:
        raise ValueError(f"K-grouped: A must be [K_total, M], B [K_total, N], k_offsets [G + 1]; got "
                         f"{list(a)}, {list(b)}, {list(o)}")
    K_total, M = a
    N = b[1]
    G = o[0] - 1
    if b[0] != K_total:
        raise ValueError(f"B has K_total = {b[0]}, A has K_total = {K_total}")
    nks, q, st = _scale_k(name, K_total), _fp8_types(), _scale_types(name)
    ptrs = _pointers((A, "A", q, (K_total, M)), (sA, "sA", st, (nks, _align4(M))), (B, "B", q, (K_total, N)),
                     (sB, "sB", st, (_cdiv(N, 128), nks)), (k_offsets, "k_offsets", _i32(), (G + 1,)),
                     (D, "D", _d_types(f32), (G, M, N)))
    _check(getattr(load(), name)(*ptrs, G, M, N, K_total, _stream(stream)))
    return D


def dg_fp8_k_grouped_gemm_tn_contiguous(A, sA, B, sB, k_offsets, D, stream=None):
    """Groups along K: A [K_total, M], B [K_total, N], k_offsets [G+1] int32 (multiples of 128),
    D [G, M, N] (bfloat16) = Σ over each group's K range."""
    return _k_grouped("dg_fp8_k_grouped_gemm_tn_contiguous", False, A, sA, B, sB, k_offsets, D, stream)


def dg_fp8_k_grouped_gemm_tn_contiguous_f32(A, sA, B, sB, k_offsets, D, stream=None):
    return _k_grouped("dg_fp8_k_grouped_gemm_tn_contiguous_f32", True, A, sA, B, sB, k_offsets, D, stream)


def dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0(A, sA, B, sB, k_offsets, D, stream=None):
    """The K-grouped GEMM with packed UE8M0 scales: sA [ceil(K_total/512), align4(M)], sB
    [ceil(N/128), ceil(K_total/512)] int32 (four K-blocks per word along K_total)."""
    return _k_grouped("dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0", False, A, sA, B, sB, k_offsets, D, stream)


def dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0_f32(A, sA, B, sB, k_offsets, D, stream=None):
    return _k_grouped("dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0_f32", True, A, sA, B, sB, k_offsets, D, stream)


@functools.cache
def _i32():
    import torch
    return (torch.int32,)


@functools.cache
def _rng_types():
    import torch
    return (torch.int64, torch.uint64)


@functools.cache
def _bf16():
    import torch
    return (torch.bfloat16, torch.int16, torch.uint16)


def _gated(name, f32, A, sA, B, sB, m_indices, H, GU, rng, p, stream):
    grouped = "contiguous" in name
    status = _bind().gated(_variant(name) + 4 * grouped, A, sA, B, sB, m_indices, H, GU, rng, p, _raw(stream))
    if status is not None:
        _check(status)
        return H
    a, b = _sizes(A, "A"), _sizes(B, "B")
    if len(a) != 2 or len(b) != (3 if grouped else 2):
        raise ValueError(f"gated projection: A must be [M, K] and B {'[G, 2I, K]' if grouped else '[2I, K]'}, "
                         f"got {list(a)} and {list(b)}")
    M, K = a
    G, N = (b[0], b[1]) if grouped else (1, b[0])
    if b[-1] != K:
        raise ValueError(f"B has K = {b[-1]}, A has K = {K}")
    if N % 2:
        raise ValueError(f"B must hold I gate rows and I up rows, got {N}")
    nks, q, st = _scale_k(name, K), _fp8_types(), _scale_types(name)
    sb = (_cdiv(N, 128), nks)
    # (of a dense call the m_indices argument is an absent optional one, and not passed on)
    pA, psA, pB, psB, pidx, pH, pGU, prng = _pointers(
        (A, "A", q, (M, K)), (sA, "sA", st, (nks, _align4(M))), (B, "B", q, b), (sB, "sB", st, (G,) + sb if grouped else sb),
        (m_indices, "m_indices" if grouped else "m_indices?", _i32(), (M,)), (H, "H", _d_types(f32), (M, N // 2)),
        (GU, "GU?", _bf16(), (M, N)), (rng, "rng?", _rng_types(), (2,)))
    f = getattr(load(), name)
    if grouped:
        _check(f(pA, psA, pB, psB, pidx, pH, pGU, prng, p, M, N, K, G, _stream(stream)))
    else:
        _check(f(pA, psA, pB, psB, pH, pGU, prng, p, M, N, K, _stream(stream)))
    return H


def dg_fp8_gemm_nt_swiglu(A, sA, B, sB, H, GU=None, rng=None, p=0.0, stream=None):
    """Gated projection H [M, I] = dropout(silu(A·Bgᵀ) · (A·Buᵀ)); B [2I, K] holds the I gate rows, then the I
    up rows (I a multiple of 128). GU (bfloat16 [M, 2I], optional) receives the pre-activations. With p > 0,
    rng is a CUDA int64 tensor {seed, offset}, read on the device."""
    return _gated("dg_fp8_gemm_nt_swiglu", False, A, sA, B, sB, None, H, GU, rng, p, stream)


def dg_fp8_gemm_nt_swiglu_f32(A, sA, B, sB, H, GU=None, rng=None, p=0.0, stream=None):
    """As dg_fp8_gemm_nt_swiglu, with H in FP32."""
    return _gated("dg_fp8_gemm_nt_swiglu_f32", True, A, sA, B, sB, None, H, GU, rng, p, stream)


def dg_fp8_gemm_nt_swiglu_ue8m0(A, sA, B, sB, H, GU=None, rng=None, p=0.0, stream=None):
    """dg_fp8_gemm_nt_swiglu with packed UE8M0 scales."""
    return _gated("dg_fp8_gemm_nt_swiglu_ue8m0", False, A, sA, B, sB, None, H, GU, rng, p, stream)


def dg_fp8_gemm_nt_swiglu_ue8m0_f32(A, sA, B, sB, H, GU=None, rng=None, p=0.0, stream=None):
    return _gated("dg_fp8_gemm_nt_swiglu_ue8m0_f32", True, A, sA, B, sB, None, H, GU, rng, p, stream)


def dg_fp8_grouped_contiguous_swiglu(A, sA, B, sB, m_indices, H, GU=None, rng=None, p=0.0, stream=None):
    """The gated projection over contiguous groups: B [G, 2I, K], row m uses expert m_indices[m] (-1: padding,
    untouched in H and GU)."""
    return _gated("dg_fp8_grouped_contiguous_swiglu", False, A, sA, B, sB, m_indices, H, GU, rng, p, stream)


def dg_fp8_grouped_contiguous_swiglu_f32(A, sA, B, sB, m_indices, H, GU=None, rng=None, p=0.0, stream=None):
    return _gated("dg_fp8_grouped_contiguous_swiglu_f32", True, A, sA, B, sB, m_indices, H, GU, rng, p, stream)


def dg_fp8_grouped_contiguous_swiglu_ue8m0(A, sA, B, sB, m_indices, H, GU=None, rng=None, p=0.0, stream=None):
    """dg_fp8_grouped_contiguous_swiglu with packed UE8M0 scales."""
    return _gated("dg_fp8_grouped_contiguous_swiglu_ue8m0", False, A, sA, B, sB, m_indices, H, GU, rng, p, stream)


def dg_fp8_grouped_contiguous_swiglu_ue8m0_f32(A, sA, B, sB, m_indices, H, GU=None, rng=None, p=0.0, stream=None):
    return _gated("dg_fp8_grouped_contiguous_swiglu_ue8m0_f32", True, A, sA, B, sB, m_indices, H, GU, rng, p, stream)


def _contig_nn(name, f32, A, sA, B, sB, m_indices, D, stream):
    status = _bind().contiguous(_variant(name) + 4, A, sA, B, sB, m_indices, D, _raw(stream))
    if status is not None:
        _check(status)
        return D
    a, b = _sizes(A, "A"), _sizes(B, "B")
    if len(a) != 2 or len(b) != 3:
        raise ValueError(f"contiguous NN: A must be [M_total, K] and B [G, K, N], got {list(a)} and {list(b)}")
    M, K = a
    G, N = b[0], b[2]
    if b[1] != K:
        raise ValueError(f"B has K = {b[1]}, A has K = {K}")
    nks, q, st = _scale_k(name, K), _fp8_types(), _scale_types(name)
    ptrs = _pointers((A, "A", q, (M, K)), (sA, "sA", st, (nks, _align4(M))), (B, "B", q, (G, K, N)),
                     (sB, "sB", st, (G, _cdiv(N, 128), nks)), (m_indices, "m_indices", _i32(), (M,)),
                     (D, "D", _d_types(f32), (M, N)))
    _check(getattr(load(), name)(*ptrs, M, N, K, G, _stream(stream)))
    return D


def dg_fp8_grouped_contiguous_nn(A, sA, B, sB, m_indices, D, stream=None):
    """Contiguous-layout grouped GEMM with B stored [G, K, N] (N contiguous; K a multiple of 128), e.g. the
    experts' input gradient dX = dY·W from the forward pass's W; sB [G, ceil(N/128), K/128]."""
    return _contig_nn("dg_fp8_grouped_contiguous_nn", False, A, sA, B, sB, m_indices, D, stream)


def dg_fp8_grouped_contiguous_nn_f32(A, sA, B, sB, m_indices, D, stream=None):
    return _contig_nn("dg_fp8_grouped_contiguous_nn_f32", True, A, sA, B, sB, m_indices, D, stream)


def dg_fp8_grouped_contiguous_nn_ue8m0(A, sA, B, sB, m_indices, D, stream=None):
    """dg_fp8_grouped_contiguous_nn with packed UE8M0 scales."""
    return _contig_nn("dg_fp8_grouped_contiguous_nn_ue8m0", False, A, sA, B, sB, m_indices, D, stream)


def dg_fp8_grouped_contiguous_nn_ue8m0_f32(A, sA, B, sB, m_indices, D, stream=None):
    return _contig_nn("dg_fp8_grouped_contiguous_nn_ue8m0_f32", True, A, sA, B, sB, m_indices, D, stream)


def _swiglu_backward(name, dH, GU, dGUr, sR, dGUc, sC, Hb, sHb, m_indices, rng, p, stream):
    status = _bind().backward(_variant(name) >> 1, dH, GU, dGUr, sR, dGUc, sC, Hb, sHb, m_indices, rng, p, _raw(stream))
    if status is not None:
        _check(status)
        return dGUr, dGUc
    h = _sizes(dH, "dH")
    if len(h) != 2:
        raise ValueError(f"dH must be [M, I], got {list(h)}")
    M, I = h
    st, q, b = _scale_types(name), _fp8_types(), _bf16()
    wM, wN = _scale_k(name, M), _scale_k(name, 2 * I)
    p_dh, p_gu, p_idx, p_rng, *forms = _pointers(
        (dH, "dH", b, h), (GU, "GU", b, (M, 2 * I)), (m_indices, "m_indices?", _i32(), (M,)), (rng, "rng?", _rng_types(), (2,)),
        (dGUr, "dGUr?", q, (M, 2 * I)), (sR, "sR?", st, (wN, _align4(M))), (dGUc, "dGUc?", q, (M, 2 * I)),
        (sC, "sC?", st, (wM, 2 * I)), (Hb, "Hb?", q, h), (sHb, "sHb?", st, (_cdiv(I, 128), wM)))
    _check(getattr(load(), name)(p_dh, p_gu, p_idx, p_rng, p, *forms, M, I, _stream(stream)))
    return dGUr, dGUc


def dg_swiglu_backward_fp8(dH, GU, dGUr=None, sR=None, dGUc=None, sC=None, Hb=None, sHb=None, m_indices=None,
                           rng=None, p=0.0, stream=None):
    """The gated projection's backward pass up to the products: from dH [M, I] and the saved GU [M, 2I]
    (bfloat16), the gradients of the pre-activations as E4M3 in one or both forms: dGUr with sR
    [2I/128, align4(M)] (A of the NN products: dX = dGU·W) and dGUc with sC [ceil(M/128), 2I] (A of the TN
    and K-grouped products: dW = dGUᵀ·X). Hb with sHb [I/128, ceil(M/128)], optional: H again in 128x128 blocks
    (B of the down projection's weight gradient). Rows with m_indices[m] < 0 count as zero. rng and p as in
    the forward call."""
    return _swiglu_backward("dg_swiglu_backward_fp8", dH, GU, dGUr, sR, dGUc, sC, Hb, sHb, m_indices, rng, p, stream)


def dg_swiglu_backward_fp8_ue8m0(dH, GU, dGUr=None, sR=None, dGUc=None, sC=None, Hb=None, sHb=None, m_indices=None,
                                 rng=None, p=0.0, stream=None):
    """dg_swiglu_backward_fp8 with power-of-two scales packed as UE8M0: sR [ceil(2I/512), align4(M)], sC
    [ceil(M/512), 2I], sHb [I/128, ceil(M/512)] int32."""
    return _swiglu_backward("dg_swiglu_backward_fp8_ue8m0", dH, GU, dGUr, sR, dGUc, sC, Hb, sHb, m_indices, rng, p, stream)


def _cast(name, X, Xr, sR, Xc, sC, Xb, sB, sBt, m_indices, stream):
    status = _bind().cast(_variant(name) >> 1, X, Xr, sR, Xc, sC, Xb, sB, sBt, m_indices, _raw(stream))
    if status is not None:
        _check(status)
        return
    x = _sizes(X, "X")
    if len(x) not in (2, 3):
        raise ValueError(f"X must be [M, N] or [G, M, N], got {list(x)}")
    M, N = x[-2:]
    g = tuple(x[:-2])
    st, q = _scale_types(name), _fp8_types()
    wM, wN, Mb, Nb = _scale_k(name, M), _scale_k(name, N), _cdiv(M, 128), _cdiv(N, 128)
    ptrs = _pointers((X, "X", _bf16(), x), (m_indices, "m_indices?", _i32(), (M,)), (Xr, "Xr?", q, x),
                     (sR, "sR?", st, g + (wN, _align4(M))), (Xc, "Xc?", q, x), (sC, "sC?", st, g + (wM, _align4(N))),
                     (Xb, "Xb?", q, x), (sB, "sB?", st, g + (Mb, wN)), (sBt, "sBt?", st, g + (Nb, wM)))
    _check(getattr(load(), name)(*ptrs, g[0] if g else 1, M, N, _stream(stream)))


def dg_cast_fp8(X, Xr=None, sR=None, Xc=None, sC=None, Xb=None, sB=None, sBt=None, m_indices=None, stream=None):
    """E4M3 casts of X (bfloat16 [M, N] or [G, M, N]) in the layouts the products read, from one read of X:
    Xr with sR [ceil(N/128), align4(M)]: 1x128 groups of each row (A of the NT and NN products);
    Xc with sC [ceil(M/128), align4(N)]: 128x1 groups of each column (A, stored [K, M], of the TN and K-grouped products);
    Xb with sB [ceil(M/128), ceil(N/128)] (B stored [N, K]) and/or sBt, its transpose (B stored [K, N]): 128x128 blocks.
    Rows with m_indices[m] < 0 count as zero."""
    _cast("dg_cast_fp8", X, Xr, sR, Xc, sC, Xb, sB, sBt, m_indices, stream)


def dg_cast_fp8_ue8m0(X, Xr=None, sR=None, Xc=None, sC=None, Xb=None, sB=None, sBt=None, m_indices=None, stream=None):
    """dg_cast_fp8 with power-of-two scales packed as UE8M0 words: sR [ceil(N/512), align4(M)], sC
    [ceil(M/512), align4(N)], sB [ceil(M/128), ceil(N/512)], sBt [ceil(N/128), ceil(M/512)] int32."""
    _cast("dg_cast_fp8_ue8m0", X, Xr, sR, Xc, sC, Xb, sB, sBt, m_indices, stream)


def dg_dropout(X, Y, rng, p, R=None, stream=None):
    """Y = R + dropout(X) (R optional), bfloat16 or float32 tensors of one shape; Y may be X or R. rng is a CUDA
    int64 tensor {seed, offset}; the mask is a function of it, p and the flat index. Backward: the same
    call on the gradient, without R."""
    status = _bind().dropout(X, R, Y, rng, p, _raw(stream))
    if status is not None:
        _check(status)
        return Y
    f32 = getattr(X, "dtype", None) in _f32()
    dt, shape = _f32() if f32 else _bf16(), _shape(X, "X")
    pX, pR, pY, prng = _pointers((X, "X", dt, shape), (R, "R?", dt, shape), (Y, "Y", dt, shape), (rng, "rng?", _rng_types(), (2,)))
    f = load().dg_dropout_f32 if f32 else load().dg_dropout_bf16
    _check(f(pX, pR, pY, prng, p, X.numel(), _stream(stream)))
    return Y


def dg_fp8_grouped_masked_swiglu(A, sA, B, sB, masked_m, H, stream=None):
    """Masked grouped GEMM fused with SwiGLU: B [G, 2I, K] (gate rows, then up rows),
    H [G, M_max, I] = silu(gate)·up over the rows m < masked_m[g]; other rows untouched."""
    return _masked("dg_fp8_grouped_masked_swiglu", False, A, sA, B, sB, masked_m, H, stream)


def dg_fp8_grouped_masked_swiglu_f32(A, sA, B, sB, masked_m, H, stream=None):
    return _masked("dg_fp8_grouped_masked_swiglu_f32", True, A, sA, B, sB, masked_m, H, stream)


def dg_fp8_grouped_masked_swiglu_fp8(A, sA, B, sB, masked_m, Hq, sH, stream=None):
    """The fused SwiGLU with H cast to FP8 for the down projection: Hq [G, M_max, I] E4M3 codes
    (uint8 or float8_e4m3fn), e4m3_rne(H · (448/amax)), and sH [G, I/128, align4(M_max)] float32, the
    dequantisation scale amax/448 of each 1x128 group of each valid row; the A and sA layouts of
    dg_fp8_grouped_masked. Rows past masked_m are
    untouched in both."""
    a, b = _sizes(A, "A"), _sizes(B, "B")
    if len(a) != 3 or len(b) != 3:
        raise ValueError(f"masked layout: A must be [G, M_max, K] and B [G, 2I, K], got {list(a)} and {list(b)}")
    G, M_max, K = a
    N = b[1]
    if b[0] != G or b[2] != K:
        raise ValueError(f"B has shape {list(b)}, expected [{G}, 2I, {K}]")
    nkb = _cdiv(K, 128)
    _expect(sA, "sA", (G, nkb, _align4(M_max)))
    _expect(sB, "sB", (G, _cdiv(N, 128), nkb))
    _expect(masked_m, "masked_m", (G,))
    _expect(Hq, "Hq", (G, M_max, N // 2))
    _expect(sH, "sH", (G, (N // 2) // 128, _align4(M_max)))
    lib = load()
    _check(lib.dg_fp8_grouped_masked_swiglu_fp8(
        _ptr(A, "A", _fp8_types()), _ptr(sA, "sA", _f32()), _ptr(B, "B", _fp8_types()), _ptr(sB, "sB", _f32()),
        _ptr(masked_m, "masked_m", _i32()), _ptr(Hq, "Hq", _fp8_types()), _ptr(sH, "sH", _f32()),
        G, M_max, N, K, _stream(stream)))
    return Hq, sH


def dg_fp8_grouped_masked_swiglu_ue8m0(A, sA, B, sB, masked_m, H, stream=None):
    """The fused SwiGLU with packed UE8M0 scales (int32 words, four K-groups each)."""
    return _masked("dg_fp8_grouped_masked_swiglu_ue8m0", False, A, sA, B, sB, masked_m, H, stream)


def dg_fp8_grouped_masked_swiglu_ue8m0_f32(A, sA, B, sB, masked_m, H, stream=None):
    return _masked("dg_fp8_grouped_masked_swiglu_ue8m0_f32", True, A, sA, B, sB, masked_m, H, stream)


def dg_transform_sf_into_ue8m0_a(sA, sA_packed, M, K, stream=None):
    """A's FP32 scales sA [ceil(K/128), align4(M)] (or [G, ...]; powers of two, zero for padding rows)
    -> packed UE8M0 words sA_packed [ceil(ceil(K/128)/4), align4(M)] (or [G, ...]) int32, on the GPU.
    A value that is not a power of two sets DG_DEV_BAD_SCALE (dg_get_device_status)."""
    import torch
    s = _sizes(sA, "sA")
    if len(s) not in (2, 3):
        raise ValueError(f"sA must be [ceil(K/128), align4(M)] or [G, ceil(K/128), align4(M)], got {list(s)}")
    G = s[0] if len(s) == 3 else 1
    nkb, ldsa = -(-K // 128), dg_get_tma_aligned_size(M, 4)
    _expect(sA, "sA", s[:-2] + (nkb, ldsa))
    _expect(sA_packed, "sA_packed", s[:-2] + (-(-nkb // 4), ldsa))
    _check(load().dg_transform_sf_into_ue8m0_a(_ptr(sA, "sA", (torch.float32,)),
                                               _ptr(sA_packed, "sA_packed", (torch.int32,)), G, M, K, _stream(stream)))


def dg_transform_sf_a_into_mn_major(sA_rows, sA, M, K, stream=None):
    """A's FP32 scales row-major sA_rows [M, ceil(K/128)] (or [G, M, ceil(K/128)]) -> the MN-major
    layout of every call, sA [ceil(K/128), align4(M)] (or [G, ...]), padding rows zero, on the GPU."""
    import torch
    s = _sizes(sA_rows, "sA_rows")
    if len(s) not in (2, 3):
        raise ValueError(f"sA_rows must be [M, ceil(K/128)] or [G, M, ceil(K/128)], got {list(s)}")
    G = s[0] if len(s) == 3 else 1
    nkb = -(-K // 128)
    _expect(sA_rows, "sA_rows", s[:-2] + (M, nkb))
    _expect(sA, "sA", s[:-2] + (nkb, dg_get_tma_aligned_size(M, 4)))
    _check(load().dg_transform_sf_a_into_mn_major(_ptr(sA_rows, "sA_rows", (torch.float32,)),
                                                  _ptr(sA, "sA", (torch.float32,)), G, M, K, _stream(stream)))


def dg_transform_sf_into_ue8m0_b(sB, sB_packed, N, K, stream=None):
    """B's FP32 scales sB [ceil(N/128), ceil(K/128)] (or [G, ...]; powers of two) -> packed UE8M0 words
    sB_packed [ceil(N/128), ceil(ceil(K/128)/4)] (or [G, ...]) int32, on the GPU. A value that is not a
    power of two sets DG_DEV_BAD_SCALE (dg_get_device_status)."""
    import torch
    s = _sizes(sB, "sB")
    if len(s) not in (2, 3):
        raise ValueError(f"sB must be [ceil(N/128), ceil(K/128)] or [G, ceil(N/128), ceil(K/128)], got {list(s)}")
    G = s[0] if len(s) == 3 else 1
    nnb, nkb = -(-N // 128), -(-K // 128)
    _expect(sB, "sB", s[:-2] + (nnb, nkb))
    _expect(sB_packed, "sB_packed", s[:-2] + (nnb, -(-nkb // 4)))
    _check(load().dg_transform_sf_into_ue8m0_b(_ptr(sB, "sB", (torch.float32,)),
                                               _ptr(sB_packed, "sB_packed", (torch.int32,)), G, N, K, _stream(stream)))


def dg_fp8_gemm_nt_ue8m0(A, sA, B, sB, D, stream=None):
    """Dense D (bfloat16) with power-of-two scales given as packed UE8M0 int32 words."""
    return _dense("dg_fp8_gemm_nt_ue8m0", False, A, sA, B, sB, D, stream)


def dg_fp8_gemm_nt_ue8m0_f32(A, sA, B, sB, D, stream=None):
    return _dense("dg_fp8_gemm_nt_ue8m0_f32", True, A, sA, B, sB, D, stream)


def dg_fp8_grouped_contiguous_ue8m0(A, sA, B, sB, m_indices, D, stream=None):
    return _contig("dg_fp8_grouped_contiguous_ue8m0", False, A, sA, B, sB, m_indices, D, stream)


def dg_fp8_grouped_contiguous_ue8m0_f32(A, sA, B, sB, m_indices, D, stream=None):
    return _contig("dg_fp8_grouped_contiguous_ue8m0_f32", True, A, sA, B, sB, m_indices, D, stream)


def dg_fp8_grouped_masked_ue8m0(A, sA, B, sB, masked_m, D, stream=None):
    return _masked("dg_fp8_grouped_masked_ue8m0", False, A, sA, B, sB, masked_m, D, stream)


def dg_fp8_grouped_masked_ue8m0_f32(A, sA, B, sB, masked_m, D, stream=None):
    return _masked("dg_fp8_grouped_masked_ue8m0_f32", True, A, sA, B, sB, masked_m, D, stream)


def dg_get_tma_aligned_size(x: int, elem_bytes: int) -> int:
    return int(load().dg_get_tma_aligned_size(x, elem_bytes))


def dg_get_mk_alignment_for_contiguous_layout() -> int:
    return int(load().dg_get_mk_alignment_for_contiguous_layout())


def dg_set_num_sms(n: int) -> None:
    load().dg_set_num_sms(int(n))


def dg_get_num_sms() -> int:
    return int(load().dg_get_num_sms())


def dg_set_cluster_split(on: bool) -> bool:
    """Allow (default) or forbid split-K inside thread-block clusters. Returns the previous value."""
    return bool(load().dg_set_cluster_split(1 if on else 0))


def dg_set_wait_limit_us(us: int) -> int:
    """Time limit of the kernels' pipeline waits in microseconds (default 2 s; < 0 restores it; 0 makes
    every wait that is not already satisfied give up, which exercises the timeout path). A launch that
    gives up sets DG_DEV_TIMEOUT; its output is undefined. Returns the previous value."""
    return int(load().dg_set_wait_limit_us(int(us)))


def dg_set_pair_b(on: bool) -> bool:
    """Allow or forbid (default) walking the tiles by pairs of CTAs that ask for the same B tiles at the same time. Returns
    the previous value; results are bit-identical either way."""
    return bool(load().dg_set_pair_b(1 if on else 0))


def _pdl(v):
    return None if v < 0 else bool(v)


def dg_set_pdl(on):
    """Launch every call with programmatic dependent launch (it may start before the previous kernel in the stream
    ends, and waits for that kernel's results before reading its inputs): True always, False never, None (the
    default) where a call is elementwise or at most one wave of tiles. Returns the previous setting, in the same
    three values, so that passing it back restores it; results are bit-identical either way."""
    return _pdl(load().dg_set_pdl(-1 if on is None else (1 if on else 0)))


def dg_get_pdl():
    """The current setting: True, False or None, as dg_set_pdl takes it."""
    return _pdl(load().dg_get_pdl())


def dg_set_tail_splits(n: int) -> int:
    """Most K ranges a tile of a last, partial wave may be cut into (1: off; <= 0: default 4).
    Returns the previous value."""
    return int(load().dg_set_tail_splits(int(n)))


def dg_get_device_status(stream=None) -> int:
    """Synchronises `stream`, reads and clears the device status word; returns its DG_DEV_* bits."""
    code = ctypes.c_int(0)
    st = load().dg_get_device_status(ctypes.byref(code), _stream(stream))
    if st not in (DG_OK, DG_ERR_DEVICE_STATUS):
        _check(st)
    return int(code.value)


def dg_last_error_string() -> str:
    return load().dg_last_error_string().decode(errors="replace")


def dg_query_config(mode: int, M: int, N: int, K: int, G: int = 1, out_f32: bool = False) -> dict:
    """Tile configuration a call would launch: mode 0 dense, 1 contiguous, 2 masked."""
    cfg = (ctypes.c_int * 6)()
    _check(load().dg_query_config(mode, M, N, K, G, 1 if out_f32 else 0, cfg))
    keys = ("block_m", "block_n", "stages", "splits", "grid", "tiles")
    return dict(zip(keys, [int(v) for v in cfg]))


def dg_query_config_ue8m0(mode: int, M: int, N: int, K: int, G: int = 1, out_f32: bool = False) -> dict:
    """Tile configuration of the packed-UE8M0 (block-scaled) calls."""
    cfg = (ctypes.c_int * 6)()
    _check(load().dg_query_config_ue8m0(mode, M, N, K, G, 1 if out_f32 else 0, cfg))
    keys = ("block_m", "block_n", "stages", "splits", "grid", "tiles")
    return dict(zip(keys, [int(v) for v in cfg]))
