"""Waits that run out in the middle of a launch: a warp ends them with one verdict, and what is in flight lands first.

With limits of a few microseconds some waits of a launch are satisfied and others give up, at any K-block and in any
role, and the lanes of a warp read the timer on both sides of the limit. Whatever happens, the launch has to end by
itself, the status word may only say DG_DEV_TIMEOUT, and the next call with the default limit has to give the
bits that it gave before. No fault, trap or hang is involved: every wait has a limit, the drains a fixed one.
"""
import numpy as np
import pytest
import torch

import dg_inputs
from _dg_testlib import bf16_sentinel, dev

pytestmark = pytest.mark.gpu

LIMITS_US = (1, 2, 3, 4, 6, 9, 14, 20, 40)


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    assert m.dg_get_device_status() == 0
    yield m
    m.dg_set_wait_limit_us(-1)
    assert m.dg_get_device_status() == 0


def _operands(M, N, K, G, ue, seed):
    a, b = dg_inputs.make_a(M, K, seed=seed, ue8m0=ue), dg_inputs.make_b(G, N, K, seed=seed, ue8m0=ue)
    sA, sB = (dg_inputs.pack_ue8m0_a(a.sA), dg_inputs.pack_ue8m0_b(b.sB)) if ue else (a.sA, b.sB)
    return dev(a.A), dev(sA), dev(b.B), dev(sB)


def _dense(dg, ue, M=640, N=2112, K=2048):
    A, sA, B, sB = _operands(M, N, K, 1, ue, 1)
    D = bf16_sentinel((M, N))
    f = dg.dg_fp8_gemm_nt_ue8m0 if ue else dg.dg_fp8_gemm_nt
    return (lambda: f(A, sA, B[0], sB[0], D)), D


def _split_k(dg, ue):
    return _dense(dg, ue, 64, 2112, 7168)


def _short_k(dg, ue):
    return _dense(dg, ue, 4096, 2112, 256)      # fewer K-blocks a tile than stages, several tiles a CTA


def _contiguous(dg, ue):
    idx = dg_inputs.contiguous_m_indices([300, 0, 520, 128])
    A, sA, B, sB = _operands(len(idx), 1024, 1536, 4, ue, 2)
    D, I = bf16_sentinel((len(idx), 1024)), dev(idx)
    f = dg.dg_fp8_grouped_contiguous_ue8m0 if ue else dg.dg_fp8_grouped_contiguous
    return (lambda: f(A, sA, B, sB, I, D)), D


def _masked(dg, ue, swiglu=False):
    G, M_max, N, K = 8, 192, 1024, 1536
    mm = dg_inputs.make_masked_m(G, M_max, seed=3)
    a, b = dg_inputs.make_masked_a(G, M_max, K, seed=3, ue8m0=ue), dg_inputs.make_b(G, N, K, seed=3, ue8m0=ue)
    sA, sB = (dg_inputs.pack_ue8m0_a(a.sA), dg_inputs.pack_ue8m0_b(b.sB)) if ue else (a.sA, b.sB)
    A, sA, B, sB, MM = dev(a.A), dev(sA), dev(b.B), dev(sB), dev(mm)
    D = bf16_sentinel((G, M_max, N // 2 if swiglu else N))
    f = getattr(dg, "dg_fp8_grouped_masked" + ("_swiglu" if swiglu else "") + ("_ue8m0" if ue else ""))
    return (lambda: f(A, sA, B, sB, MM, D)), D


def _masked_swiglu(dg, ue):
    return _masked(dg, ue, True)


def _gated(dg, ue):
    M, N, K = 640, 1024, 2048
    A, sA, B, sB = _operands(M, N, K, 1, ue, 4)
    H, GU = bf16_sentinel((M, N // 2)), bf16_sentinel((M, N))
    f = dg.dg_fp8_gemm_nt_swiglu_ue8m0 if ue else dg.dg_fp8_gemm_nt_swiglu
    return (lambda: f(A, sA, B[0], sB[0], H, GU=GU)), H


def _k_grouped(dg, ue):
    M, N, off = 512, 1024, np.array([0, 1024, 1024, 3072], np.int32)
    K = int(off[-1])
    a, b = dg_inputs.make_a(M, K, seed=5, ue8m0=ue), dg_inputs.make_b(1, N, K, seed=5, ue8m0=ue)
    A, B, O = dev(np.ascontiguousarray(a.A.T)), dev(np.ascontiguousarray(b.B[0].T)), dev(off)
    sA, sB = (dev(dg_inputs.pack_ue8m0_a(a.sA)), dev(dg_inputs.pack_ue8m0_b(b.sB)[0])) if ue else (dev(a.sA), dev(b.sB[0]))
    D = bf16_sentinel((len(off) - 1, M, N))
    f = dg.dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0 if ue else dg.dg_fp8_k_grouped_gemm_tn_contiguous
    return (lambda: f(A, sA, B, sB, O, D)), D


FORMS = {f.__name__[1:]: f for f in (_dense, _split_k, _short_k, _contiguous, _masked, _masked_swiglu, _gated, _k_grouped)}


@pytest.mark.parametrize("ue", [False, True], ids=["fp32", "ue8m0"])
@pytest.mark.parametrize("form", FORMS)
def test_waits_that_give_up_midway_end_the_launch(dg, form, ue):
    call, out = FORMS[form](dg, ue)
    call()
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0
    ref = out.clone()
    for limit in LIMITS_US:
        for _ in range(5):
            prev = dg.dg_set_wait_limit_us(limit)
            try:
                call()
                status = dg.dg_get_device_status()
            finally:
                dg.dg_set_wait_limit_us(prev)
            assert status in (0, dg.DG_DEV_TIMEOUT), f"status 0x{status:x} with a limit of {limit} us"
            if status == 0:
                assert torch.equal(out.view(torch.int8), ref.view(torch.int8)), "a launch that reported no timeout differs"
        out.view(torch.int8).fill_(-1)
        call()
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == 0
        assert torch.equal(out.view(torch.int8), ref.view(torch.int8)), f"the call after limits of {limit} us differs"


@pytest.mark.parametrize("ue", [False, True], ids=["fp32", "ue8m0"])
def test_a_limit_of_zero_with_every_load_already_issued(dg, ue):
    """Two K-blocks a tile: the producer has issued all its loads, and waits for nothing, when the others give up."""
    call, out = _dense(dg, ue, 128, 2112, 256)
    call()
    torch.cuda.synchronize()
    assert dg.dg_get_device_status() == 0
    ref = out.clone()
    for _ in range(20):
        prev = dg.dg_set_wait_limit_us(0)
        try:
            call()
            assert dg.dg_get_device_status() == dg.DG_DEV_TIMEOUT
        finally:
            dg.dg_set_wait_limit_us(prev)
        out.view(torch.int8).fill_(-1)
        call()
        torch.cuda.synchronize()
        assert dg.dg_get_device_status() == 0
        assert torch.equal(out.view(torch.int8), ref.view(torch.int8))
