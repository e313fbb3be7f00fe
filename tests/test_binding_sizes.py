"""Extents that the C entry points' int cannot hold are refused (they used to be passed on modulo 2^32: a cast of 2^32 rows
returned without an error and without writing anything). Meta tensors: no memory is needed to ask."""
import pytest
import torch

import moe_grouped_gemm_e4m3_gb300 as dg

BIG = 2 ** 32


def _t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="meta")


def u8(*s):
    return _t(torch.uint8, *s)


def f32(*s):
    return _t(torch.float32, *s)


def i32(*s):
    return _t(torch.int32, *s)


def bf16(*s):
    return _t(torch.bfloat16, *s)


CALLS = {
    "dg_cast_fp8": dict(X=bf16(BIG, 16), Xr=u8(BIG, 16), sR=f32(1, BIG)),
    "dg_cast_fp8_ue8m0": dict(X=bf16(BIG, 1, 16), Xb=u8(BIG, 1, 16), sB=i32(BIG, 1, 1)),
    "dg_swiglu_backward_fp8": dict(dH=bf16(BIG, 128), GU=bf16(BIG, 256), dGUr=u8(BIG, 256), sR=f32(2, BIG)),
    "dg_fp8_gemm_nt": dict(A=u8(BIG, 128), sA=f32(1, BIG), B=u8(64, 128), sB=f32(1, 1), D=bf16(BIG, 64)),
    "dg_fp8_gemm_nt_acc_f32": dict(A=u8(BIG, 128), sA=f32(1, BIG), B=u8(64, 128), sB=f32(1, 1), C=f32(BIG, 64), D=f32(BIG, 64)),
    "dg_fp8_gemm_nn": dict(A=u8(BIG, 128), sA=f32(1, BIG), B=u8(128, 64), sB=f32(1, 1), D=bf16(BIG, 64), M=BIG, N=64, K=128),
    "dg_fp8_gemm_nt_swiglu": dict(A=u8(BIG, 128), sA=f32(1, BIG), B=u8(256, 128), sB=f32(2, 1), H=bf16(BIG, 128)),
    "dg_fp8_grouped_contiguous": dict(A=u8(BIG, 128), sA=f32(1, BIG), B=u8(2, 64, 128), sB=f32(2, 1, 1), m_indices=i32(BIG), D=bf16(BIG, 64)),
    "dg_fp8_grouped_contiguous_nn": dict(A=u8(BIG, 128), sA=f32(1, BIG), B=u8(2, 128, 64), sB=f32(2, 1, 1), m_indices=i32(BIG), D=bf16(BIG, 64)),
    "dg_fp8_grouped_masked": dict(A=u8(1, BIG, 128), sA=f32(1, 1, BIG), B=u8(1, 64, 128), sB=f32(1, 1, 1), masked_m=i32(1), D=bf16(1, BIG, 64)),
    "dg_fp8_k_grouped_gemm_tn_contiguous": dict(A=u8(BIG, 64), sA=f32(BIG // 128, 64), B=u8(BIG, 64), sB=f32(1, BIG // 128), k_offsets=i32(2),
                                                D=bf16(1, 64, 64)),
    "dg_transform_sf_into_ue8m0_b": dict(sB=f32(BIG, 1, 1), sB_packed=i32(BIG, 1, 1), N=128, K=128),
}


@pytest.mark.parametrize("call", CALLS)
def test_extents_past_32_bits_are_refused(call):
    with pytest.raises(ValueError, match=r"2\^31"):
        getattr(dg, call)(**CALLS[call])


def test_dropout_takes_any_number_of_elements():
    x = bf16(BIG + 8)
    with pytest.raises(ValueError, match="CUDA tensor"):       # (past the sizes: only the place is wrong)
        dg.dg_dropout(x, x, None, 0.0)
