"""The operators around the experts' products without a GPU: the binding refuses wrong shapes, types and places before it
takes a pointer, and the library's own checks refuse bad arguments before any CUDA call."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_e4m3_gb300 as dg

M, N, T, E, k, K, I = 70, 272, 5, 6, 2, 288, 256


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(s)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


CALLS = {
    "dg_residual_norm": dict(X=bf(M, N), W=f32(N), B=bf(M, N), w_after=f32(N), gate=f32(M), scale=f32(N), R=bf(M, N), Y=bf(M, N),
                             Yq=u8(M, N), sY=f32(3, 72), rstd=f32(M), rstd_after=f32(M)),
    "dg_residual_norm_ue8m0": dict(X=f32(M, N), W=f32(N), Yq=u8(M, N), sY=i32(1, 72)),
    "dg_residual_norm_backward": dict(dY=bf(M, N), R=bf(M, N), rstd=f32(M), W=f32(N), dR=bf(M, N), B=bf(M, N), rstd_after=f32(M),
                                      w_after=f32(N), gate=f32(M), scale=f32(N), dX=bf(M, N), dB=bf(M, N), dW=f32(N),
                                      dw_after=f32(N), dgate=f32(M), dscale=f32(N)),
    "dg_route_topk": dict(logits=f32(T, E), ids=i32(T, k), weights=f32(T, k), bias=f32(E)),
    "dg_route_topk_backward": dict(dweights=f32(T, k), logits=bf(T, E), ids=i32(T, k), dlogits=bf(T, E)),
    "dg_fp8_moe_swiglu": dict(A=u8(T, K), sA=f32(3, 8), W1=u8(E, 2 * I, K), sW1=f32(E, 4, 3), W2=u8(E, K, I), sW2=f32(E, 3, 2),
                              topk_ids=i32(T, k), topk_weights=f32(T, k), Y=bf(T, K)),
    "dg_fp8_moe_swiglu_ue8m0": dict(A=u8(T, K), sA=i32(1, 8), W1=u8(E, 2 * I, K), sW1=i32(E, 4, 1), W2=u8(E, K, I), sW2=i32(E, 3, 1),
                                    topk_ids=i32(T, k), topk_weights=f32(T, k), Y=bf(T, K)),
    "dg_fp8_moe_swiglu_mxfp4": dict(A=u8(T, K), sA=f32(3, 8), W1=u8(E, 2 * I, K // 2), sW1=u8(E, 2 * I, K // 32), W2=u8(E, K, I // 2),
                                    sW2=u8(E, K, I // 32), topk_ids=i32(T, k), topk_weights=f32(T, k), Y=bf(T, K)),
    "dg_fp8_mxfp4_gemm_nt": dict(A=u8(T, K), sA=f32(3, 8), B=u8(N, K // 2), sB=u8(N, K // 32), D=bf(T, N)),
    "dg_fp8_mxfp4_gemm_nt_f32": dict(A=u8(T, K), sA=f32(3, 8), B=u8(N, K // 2), sB=u8(N, K // 32), D=f32(T, N)),
}
NAMES = [(c, a) for c, args in CALLS.items() for a in args]


@pytest.mark.parametrize("call", CALLS)
def test_well_shaped_arguments_stop_at_their_place(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        getattr(dg, call)(**CALLS[call])


@pytest.mark.parametrize("call,arg", NAMES)
def test_wrong_shapes_are_refused(call, arg):
    t = CALLS[call][arg]
    for bad in (torch.cat([t, t[:1]], 0), t.reshape(-1)[: t.numel() - 1], t[..., :-1]):
        if bad.shape == t.shape:
            continue
        with pytest.raises((ValueError, TypeError), match=r"shape|expected|must be|groups of"):
            getattr(dg, call)(**{**CALLS[call], arg: bad})


@pytest.mark.parametrize("call,arg", NAMES)
def test_wrong_types_and_things_that_are_no_tensors_are_refused(call, arg):
    for bad in ([1.0, 2.0], CALLS[call][arg].to(torch.float64)):
        with pytest.raises((TypeError, ValueError), match="torch.Tensor|dtype|CUDA tensor"):
            getattr(dg, call)(**{**CALLS[call], arg: bad})


def test_workspaces_are_checked_like_any_tensor(monkeypatch):
    """Their type, their place and their device, which has to be the current one."""
    monkeypatch.setattr(dg, "_torch", lambda: torch)      # (without its start of the driver)
    for bad in ([1], torch.zeros(8), u8(8)):
        with pytest.raises((TypeError, ValueError), match="workspace must be a torch.Tensor|workspace has dtype|workspace must be a CUDA tensor"):
            dg._workspace(8, bad, None)

    class Elsewhere:
        dtype, shape, is_cuda, device = torch.uint8, (64,), True, torch.device("cuda", 1)
        is_contiguous, data_ptr, numel = lambda s: True, lambda s: X0, lambda s: 64

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1"):
        dg._workspace(8, Elsewhere(), None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert dg._workspace(8, Elsewhere(), None)[1:] == (X0, 64)


def test_scores_have_names():
    with pytest.raises(ValueError, match="softmax"):
        dg.dg_route_topk(**CALLS["dg_route_topk"], score="tanh")


def _p(*a):
    return [ctypes.c_void_p(x) for x in a]


X0 = 0x100000     # never dereferenced


def _at(i):
    return X0 + i * 0x1000000


INVALID, ALIGN, UNSUPPORTED, OK = dg.DG_ERR_INVALID_ARG, dg.DG_ERR_ALIGNMENT, dg.DG_ERR_UNSUPPORTED, dg.DG_OK


def test_the_library_refuses_norms():
    lib = dg.load()

    def norm(X=_at(0), B=_at(1), wa=X0, gate=X0, scale=X0, W=X0, eps=1e-6, R=_at(2), Y=_at(3), Yq=_at(4), sY=_at(5), rstd=X0, ra=X0,
             M=16, N=128):
        return lib.dg_residual_norm_bf16(*_p(X, B, wa, gate, scale, W), eps, *_p(R, Y, Yq, sY, rstd, ra), M, N, None)

    assert norm(X=None) == INVALID and norm(M=-1) == INVALID and norm(N=-1) == INVALID
    assert norm(M=0) == OK and norm(N=0) == OK and norm(N=16385) == UNSUPPORTED and norm(M=(1 << 31) - 1) == UNSUPPORTED
    assert norm(eps=-1.0) == INVALID and norm(eps=float("nan")) == INVALID and norm(eps=float("inf")) == INVALID
    assert norm(B=None) == INVALID and norm(B=None, wa=None, gate=None, scale=None, ra=None) == INVALID   # R without B
    assert norm(wa=None) == INVALID                              # rstd_after without the norm after
    assert norm(W=None) == INVALID                               # Y without W
    assert norm(R=None, Y=None, Yq=None, sY=None, rstd=None) == INVALID
    assert norm(sY=None) == INVALID and norm(Yq=None) == INVALID and norm(N=120) == ALIGN and norm(Yq=_at(4) + 8) == ALIGN
    assert norm(X=_at(0) + 1) == ALIGN and norm(W=X0 + 2) == ALIGN and norm(gate=X0 + 1) == ALIGN
    assert norm(R=_at(0) + 2) == INVALID and norm(R=_at(1) + 128) == INVALID and norm(Y=_at(2)) == INVALID and norm(Yq=_at(0)) == INVALID
    assert norm(Y=_at(0) - 16) == INVALID

    def back(dY=_at(0), dR=_at(1), R=_at(2), B=_at(3), W=X0, wa=X0, gate=X0, scale=X0, rstd=X0, ra=X0, dX=_at(4), dB=_at(5), dW=X0, dwa=X0,
             dg_=X0, ds=X0, ws=_at(6), size=1 << 40, M=16, N=128):
        return lib.dg_residual_norm_backward_f32(*_p(dY, dR, R, B, W, wa, gate, scale, rstd, ra, dX, dB, dW, dwa, dg_, ds, ws), size, M, N, None)

    assert back(M=-1) == INVALID and back(N=20000) == UNSUPPORTED and back(N=0) == OK
    assert back(dY=None, dR=None) == INVALID and back(dY=None) == INVALID and back(R=None) == INVALID and back(rstd=None) == INVALID
    assert back(W=None) == INVALID and back(B=None) == INVALID and back(ra=None) == INVALID
    assert back(wa=None) == INVALID and back(gate=None) == INVALID and back(scale=None) == INVALID
    assert back(dX=None, dB=None, dW=None, dwa=None, dg_=None, ds=None) == INVALID
    assert back(ws=None) == INVALID and back(size=100) == INVALID and back(ws=_at(6) + 8) == ALIGN
    assert back(dX=_at(0) + 4) == INVALID and back(dB=_at(4)) == INVALID and back(dX=_at(0) + 2) == ALIGN and back(dW=X0 + 1) == ALIGN


def test_the_norm_s_workspace_is_a_function_of_the_sizes():
    w = dg.dg_residual_norm_backward_workspace
    assert w(0, 128) == 0 and w(8192, 0) == 0 and w(1, 128) == 2 * 128 * 4 and w(7, 2112) == 7 * 2 * 2112 * 4
    assert w(1 << 20, 7168) == 152 * 2 * 7168 * 4 == w(1 << 24, 7168)
    with pytest.raises(ValueError, match="2\\^31"):
        w(1 << 32, 128)


def test_the_library_refuses_routes():
    lib = dg.load()

    def route(l=_at(0), b=X0, ids=_at(1), w=_at(2), score=0, factor=1.0, T=4, E=8, k=2):
        return lib.dg_route_topk_f32(*_p(l, b, ids, w), score, 1, factor, T, E, k, None)

    assert route(l=None) == INVALID and route(ids=None) == INVALID and route(w=None) == INVALID and route(T=-1) == INVALID
    assert route(E=0) == INVALID and route(k=0) == INVALID and route(k=9) == INVALID and route(score=2) == INVALID
    assert route(T=(1 << 31) - 1) == UNSUPPORTED and route(E=1025) == UNSUPPORTED and route(E=64, k=33) == UNSUPPORTED and route(T=0) == OK
    assert route(factor=float("nan")) == INVALID and route(factor=1e300) == INVALID
    assert route(l=_at(0) + 2) == ALIGN and route(b=X0 + 2) == ALIGN and route(ids=_at(1) + 1) == ALIGN
    assert lib.dg_route_topk_bf16(*_p(_at(0) + 1, None, _at(1), _at(2)), 0, 1, 1.0, 4, 8, 2, None) == ALIGN

    def back(dw=_at(0), l=_at(1), ids=_at(2), dl=_at(3), T=4):
        return lib.dg_route_topk_backward_f32(*_p(dw, l, ids, dl), 1, 0, 1.0, T, 8, 2, None)

    assert back(dw=None) == INVALID and back(l=None) == INVALID and back(ids=None) == INVALID and back(dl=None) == INVALID
    assert back(dl=_at(1) + 4) == INVALID and back(T=0) == OK


def test_the_library_refuses_products_of_few_tokens():
    lib = dg.load()

    def moe(name="", A=_at(0), sA=X0, W1=_at(1), s1=X0, W2=_at(2), s2=X0, ids=X0, w=X0, Y=_at(3), ws=_at(4), size=1 << 40, T=4, k=2, E=8, K=256,
            I=128, N=64):
        return getattr(lib, "dg_fp8_moe_swiglu" + name)(*_p(A, sA, W1, s1, W2, s2, ids, w, Y, ws), size, T, k, E, K, I, N, None)

    for name in ("", "_f32", "_ue8m0", "_ue8m0_f32", "_mxfp4", "_mxfp4_f32"):
        for null in ("A", "sA", "W1", "s1", "W2", "s2", "ids", "w", "Y", "ws"):
            assert moe(name, **{null: None}) == INVALID, null
        for off in ("A", "W1", "W2", "ws"):
            assert moe(name, **{off: _at(1) + 8}) == ALIGN, off
        for off in ("sA", "s1", "s2", "ids", "w"):
            assert moe(name, **{off: X0 + 2}) == ALIGN, off
        assert moe(name, Y=_at(3) + 1) == ALIGN and moe(name, T=-1) == INVALID and moe(name, T=0) == OK and moe(name, N=0) == OK
        assert moe(name, k=0) == INVALID and moe(name, E=0) == INVALID and moe(name, K=0) == INVALID and moe(name, I=0) == INVALID
        assert moe(name, k=33) == UNSUPPORTED and moe(name, E=1025) == UNSUPPORTED and moe(name, T=1 << 30, k=32) == UNSUPPORTED and moe(name, T=1 << 28, k=8) == UNSUPPORTED and moe(name, E=1024, I=1 << 20) == UNSUPPORTED
        assert moe(name, I=192) == ALIGN and moe(name, N=72) == ALIGN and moe(name, K=264) == ALIGN
        assert moe(name, size=100) == INVALID
    assert moe("_mxfp4", K=272) == ALIGN
    assert dg.dg_fp8_moe_workspace(0, 8, 128) == 0 and dg.dg_fp8_moe_workspace(1, 8, 128) == 8 * (128 * 5 + 4)

    def four(A=_at(0), sA=X0, B=_at(1), sB=X0, D=_at(2), M=4, N=64, K=256, name=""):
        return getattr(lib, "dg_fp8_mxfp4_gemm_nt" + name)(*_p(A, sA, B, sB, D), M, N, K, None)

    for name in ("", "_f32"):
        for null in ("A", "sA", "B", "sB", "D"):
            assert four(name=name, **{null: None}) == INVALID
        assert four(name=name, K=272) == ALIGN and four(name=name, N=60) == ALIGN and four(name=name, K=0) == INVALID
        assert four(name=name, M=-1) == INVALID and four(name=name, M=0) == OK and four(name=name, N=0) == OK
        assert four(name=name, A=_at(0) + 8) == ALIGN and four(name=name, sB=X0 + 1) == ALIGN and four(name=name, D=_at(2) + 1) == ALIGN
