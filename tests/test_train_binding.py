"""The training operators without a GPU: the binding refuses wrong shapes, types and places before it takes
a pointer, and the library's own checks refuse bad arguments before any CUDA call."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_e4m3_gb300 as dg

M, I, K, G = 70, 128, 272, 3


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(s)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


CALLS = {
    "dg_fp8_gemm_nt_swiglu": dict(A=u8(M, K), sA=f32(3, 72), B=u8(2 * I, K), sB=f32(2, 3), H=bf16(M, I), GU=bf16(M, 2 * I)),
    "dg_fp8_gemm_nt_swiglu_f32": dict(A=u8(M, K), sA=f32(3, 72), B=u8(2 * I, K), sB=f32(2, 3), H=f32(M, I)),
    "dg_fp8_gemm_nt_swiglu_ue8m0": dict(A=u8(M, K), sA=i32(1, 72), B=u8(2 * I, K), sB=i32(2, 1), H=bf16(M, I)),
    "dg_fp8_grouped_contiguous_swiglu": dict(A=u8(M, K), sA=f32(3, 72), B=u8(G, 2 * I, K), sB=f32(G, 2, 3), m_indices=i32(M),
                                             H=bf16(M, I), GU=bf16(M, 2 * I)),
    "dg_fp8_grouped_contiguous_nn": dict(A=u8(M, 256), sA=f32(2, 72), B=u8(G, 256, K), sB=f32(G, 3, 2), m_indices=i32(M), D=bf16(M, K)),
    "dg_swiglu_backward_fp8": dict(dH=bf16(M, I), GU=bf16(M, 2 * I), dGUr=u8(M, 2 * I), sR=f32(2, 72), dGUc=u8(M, 2 * I),
                                   sC=f32(1, 2 * I), Hb=u8(M, I), sHb=f32(1, 1), m_indices=i32(M)),
    "dg_swiglu_backward_fp8_ue8m0": dict(dH=bf16(M, I), GU=bf16(M, 2 * I), dGUr=u8(M, 2 * I), sR=i32(1, 72)),
    "dg_cast_fp8": dict(X=bf16(M, K), Xr=u8(M, K), sR=f32(3, 72), Xc=u8(M, K), sC=f32(1, K), Xb=u8(M, K), sB=f32(1, 3), sBt=f32(3, 1),
                        m_indices=i32(M)),
    "dg_cast_fp8_ue8m0": dict(X=bf16(G, M, K), Xr=u8(G, M, K), sR=i32(G, 1, 72), Xb=u8(G, M, K), sBt=i32(G, 3, 1)),
    "dg_dropout": dict(X=bf16(M, K), Y=bf16(M, K), rng=torch.zeros(2, dtype=torch.int64), p=0.1, R=bf16(M, K)),
}
NAMES = [(c, a) for c, args in CALLS.items() for a in args if a != "p"]


@pytest.mark.parametrize("call", CALLS)
def test_well_shaped_arguments_stop_at_their_place(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        getattr(dg, call)(**CALLS[call])


@pytest.mark.parametrize("call,arg", NAMES)
def test_wrong_shapes_are_refused(call, arg):
    t = CALLS[call][arg]
    for bad in (torch.cat([t, t[:1]], 0), t.reshape(-1)[: t.numel() - 1]):
        if bad.shape == t.shape:
            continue
        with pytest.raises((ValueError, TypeError), match=r"shape|expected|must be|has K|must hold"):
            getattr(dg, call)(**{**CALLS[call], arg: bad})


@pytest.mark.parametrize("call,arg", NAMES)
def test_things_that_are_no_tensors_are_refused(call, arg):
    with pytest.raises(TypeError, match="torch.Tensor"):
        getattr(dg, call)(**{**CALLS[call], arg: [1.0, 2.0]})


def _p(*a):
    return [ctypes.c_void_p(x) for x in a]


def test_the_library_refuses_before_any_cuda_call():
    lib, x = dg.load(), 0x10000     # never dereferenced
    ok = dict(invalid=dg.DG_ERR_INVALID_ARG, align=dg.DG_ERR_ALIGNMENT)

    def gated(A=x, sA=x, B=x, sB=x, H=x, GU=None, rng=None, p=0.0, M=16, N=256, K=128):
        return lib.dg_fp8_gemm_nt_swiglu(*_p(A, sA, B, sB, H, GU, rng), p, M, N, K, None)

    assert gated(A=None) == ok["invalid"] and gated(H=None) == ok["invalid"]
    assert gated(N=128) == ok["align"] and gated(K=120) == ok["align"] and gated(GU=x + 8) == ok["align"]
    assert gated(p=0.1) == ok["invalid"] and gated(p=1.0, rng=x) == ok["invalid"] and gated(p=-1.0, rng=x) == ok["invalid"]
    assert gated(p=float("nan"), rng=x) == ok["invalid"] and gated(p=0.1, rng=x + 4) == ok["align"]
    assert gated(M=-1) == ok["invalid"] and gated(M=0) == dg.DG_OK and gated(K=0) == ok["invalid"]

    def contiguous(idx=x, G=2, N=256):
        return lib.dg_fp8_grouped_contiguous_swiglu(*_p(x, x, x, x, idx, x, None, None), 0.0, 128, N, 128, G, None)

    assert contiguous(idx=None) == ok["invalid"] and contiguous(N=384) == ok["align"] and contiguous(G=0) == dg.DG_OK

    def nn(idx=x, N=64, K=256, G=2):
        return lib.dg_fp8_grouped_contiguous_nn(*_p(x, x, x, x, idx, x), 128, N, K, G, None)

    assert nn(idx=None) == ok["invalid"] and nn(N=72) == ok["align"] and nn(K=192) == ok["align"]
    assert nn(N=1 << 20, K=1 << 20, G=1 << 14) == dg.DG_ERR_UNSUPPORTED

    def backward(dH=x, GU=x, idx=None, rng=None, p=0.0, q=x, s=x, qc=None, sc=None, M=16, I=128):
        return lib.dg_swiglu_backward_fp8(*_p(dH, GU, idx, rng), p, *_p(q, s, qc, sc, None, None), M, I, None)

    assert backward(dH=None) == ok["invalid"] and backward(q=None, s=None) == ok["invalid"] and backward(s=None) == ok["invalid"]
    assert backward(sc=x) == ok["invalid"] and backward(I=96) == ok["align"] and backward(dH=x + 2) == ok["align"]
    assert backward(q=x + 8) == ok["align"] and backward(s=x + 2) == ok["align"] and backward(p=0.1) == ok["invalid"]
    assert backward(M=0) == dg.DG_OK

    def cast(X=x, idx=None, q=x, s=x, G=1, M=16, N=128):
        return lib.dg_cast_fp8(*_p(X, idx, q, s, None, None, None, None, None), G, M, N, None)

    assert cast(X=None) == ok["invalid"] and cast(q=None, s=None) == ok["invalid"] and cast(q=None) == ok["invalid"]
    assert cast(N=120) == ok["align"] and cast(X=x + 8) == ok["align"] and cast(idx=x, G=2) == ok["invalid"]
    assert cast(M=0) == dg.DG_OK and cast(G=1 << 20, M=1 << 20) == dg.DG_ERR_UNSUPPORTED

    def drop(X=x, R=None, Y=x + 4096, rng=x, p=0.1, n=64):
        return lib.dg_dropout_bf16(*_p(X, R, Y, rng), p, n, None)

    assert drop(X=None) == ok["invalid"] and drop(n=-1) == ok["invalid"] and drop(n=0) == dg.DG_OK
    assert drop(Y=x + 64) == ok["invalid"] and drop(X=x + 1) == ok["align"] and drop(p=0.9999999) == ok["invalid"]
    assert lib.dg_dropout_f32(*_p(x + 2, None, x + 4096, x), 0.1, 64, None) == ok["align"]


def test_tn_takes_any_k_and_the_others_do_not():
    lib, x = dg.load(), 0x10000
    for name in ("dg_fp8_gemm_nn", "dg_fp8_gemm_tt", "dg_fp8_gemm_nt"):
        assert getattr(lib, name)(*_p(x, x, x, x, x), 16, 64, 130, None) == dg.DG_ERR_ALIGNMENT
    assert lib.dg_fp8_gemm_tn(*_p(x, x, x, x, x), 24, 64, 130, None) == dg.DG_ERR_ALIGNMENT      # M % 16 still holds
