"""dg_set_num_sms holds for every operator: no launch has more CTAs than the SMs it may use, and the bits do not change.

The grids are read from torch's profiler. A cap smaller than the problem also sends the persistent kernels through several
tiles a CTA, with inputs copied ahead and buffers used again, at sizes that are quick to check.
"""
import json

import pytest
import torch

pytestmark = pytest.mark.gpu

M, I, K = 700, 384, 512


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield m
    m.dg_set_num_sms(0)
    assert m.dg_get_device_status() == 0


def _cdiv(a, b):
    return -(-a // b)


def _gen():
    return torch.Generator(device="cuda").manual_seed(9)


def _rng():
    return torch.tensor([7, 1], dtype=torch.int64, device="cuda")


def _scale(ue, *shape):
    return torch.zeros(shape, dtype=torch.int32 if ue else torch.float32, device="cuda")


def _code(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


def _groups(n, ue):
    return _cdiv(n, 512) if ue else _cdiv(n, 128)


def _holes(rows):
    """Row indices with padding in other places of every tile."""
    r = torch.arange(rows, device="cuda")
    return torch.where((r * 7 + r // 128 * 3) % 11 < 2, -1, 0).to(torch.int32)


def _few(dg, ue, tokens=9):
    q = lambda *s: (torch.rand(*s, generator=_gen(), device="cuda") * 2 - 1).to(torch.float8_e4m3fn)  # noqa: E731
    A, B, sA, sB = q(tokens, K), q(2 * I, K), _scale(ue, _groups(K, ue), 4 * _cdiv(tokens, 4)), _scale(ue, 2 * I // 128, _groups(K, ue))
    for s in (sA, sB):
        s.fill_(0x7F7E7F80 if ue else 0.5)
    H, GU = (torch.zeros(tokens, n, dtype=torch.bfloat16, device="cuda") for n in (I, 2 * I))
    f = dg.dg_fp8_gemm_nt_swiglu_ue8m0 if ue else dg.dg_fp8_gemm_nt_swiglu
    return lambda: f(A, sA, B, sB, H, GU=GU, rng=_rng_of(H), p=0.1), [H, GU]


_RNG = {}


def _rng_of(t):
    return _RNG.setdefault(t.device, _rng())


def _one(dg, ue):
    return _few(dg, ue, 1)


def _dropout(dg, ue):
    n = 100003 if ue else 65536          # (odd and FP32, or whole and BF16 with the residual)
    dt = torch.float32 if ue else torch.bfloat16
    x, r = (torch.randn(n, generator=_gen(), device="cuda").to(dt) for _ in range(2))
    y = torch.empty_like(x)
    return lambda: dg.dg_dropout(x, y, _rng_of(x), 0.2, R=None if ue else r), [y]


def _cast(dg, ue):
    x = torch.randn(M, K + 16, generator=_gen(), device="cuda").bfloat16()
    N = x.shape[1]
    o = dict(Xr=_code(M, N), sR=_scale(ue, _groups(N, ue), M), Xc=_code(M, N), sC=_scale(ue, _groups(M, ue), N), Xb=_code(M, N),
             sB=_scale(ue, _cdiv(M, 128), _groups(N, ue)), sBt=_scale(ue, _cdiv(N, 128), _groups(M, ue)))
    f = dg.dg_cast_fp8_ue8m0 if ue else dg.dg_cast_fp8
    return lambda: f(x, m_indices=_holes(M), **o), list(o.values())


def _cast_weights(dg, ue):
    x = torch.randn(3, 300, 256, generator=_gen(), device="cuda").bfloat16()
    o = dict(Xb=_code(3, 300, 256), sB=_scale(ue, 3, 3, _groups(256, ue)), sBt=_scale(ue, 3, 2, _groups(300, ue)))
    f = dg.dg_cast_fp8_ue8m0 if ue else dg.dg_cast_fp8
    return lambda: f(x, **o), list(o.values())


def _backward(dg, ue):
    dh, gu = (torch.randn(M, n, generator=_gen(), device="cuda").bfloat16() for n in (I, 2 * I))
    o = dict(dGUr=_code(M, 2 * I), sR=_scale(ue, _groups(2 * I, ue), M), dGUc=_code(M, 2 * I), sC=_scale(ue, _groups(M, ue), 2 * I),
             Hb=_code(M, I), sHb=_scale(ue, I // 128, _groups(M, ue)))
    f = dg.dg_swiglu_backward_fp8_ue8m0 if ue else dg.dg_swiglu_backward_fp8
    return lambda: f(dh, gu, m_indices=_holes(M), rng=_rng_of(dh), p=0.1, **o), list(o.values())


def _scales(dg, ue):
    """The conversions of FP32 scales, of A (row-major, then packed) and of B."""
    pow2 = lambda *s: torch.randint(-9, 9, s, generator=_gen(), device="cuda").float().exp2()  # noqa: E731
    a, b = pow2(3, M, 9), pow2(3, 70, 37)
    major, pa, pb = torch.zeros(3, 9, M, device="cuda"), _scale(True, 3, 3, M), _scale(True, 3, 70, 10)

    def call():
        dg.dg_transform_sf_a_into_mn_major(a, major, M, 9 * 128)
        dg.dg_transform_sf_into_ue8m0_a(major, pa, M, 9 * 128)
        dg.dg_transform_sf_into_ue8m0_b(b, pb, 70 * 128, 37 * 128)
    return call, [major, pa, pb]


OPS = {f.__name__[1:]: f for f in (_one, _few, _dropout, _cast, _cast_weights, _backward, _scales)}


def _grids(call, tmp_path):
    """The number of CTAs of each of the library's launches in one call."""
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    path = str(tmp_path / "trace.json")
    prof.export_chrome_trace(path)
    with open(path) as f:
        events = json.load(f)["traceEvents"]
    grids = [e["args"]["grid"] for e in events if e.get("cat") == "kernel" and "dg::" in e.get("name", "")]
    return [g[0] * g[1] * g[2] for g in grids]


@pytest.mark.parametrize("ue", [False, True], ids=["fp32", "ue8m0"])
@pytest.mark.parametrize("op", OPS)
def test_a_cap_changes_no_bits(dg, op, ue):
    call, outs = OPS[op](dg, ue)
    call()
    want = [o.clone() for o in outs]
    for cap in (1, 2, 5, 37):
        dg.dg_set_num_sms(cap)
        try:
            for o in outs:
                o.view(torch.uint8).fill_(0xFF)
            call()
        finally:
            dg.dg_set_num_sms(0)
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.uint8), w.view(torch.uint8)), f"a cap of {cap} SMs changes the result"


@pytest.mark.parametrize("ue", [False, True], ids=["fp32", "ue8m0"])
@pytest.mark.parametrize("op", OPS)
def test_a_cap_bounds_the_grid(dg, op, ue, tmp_path):
    call, _ = OPS[op](dg, ue)
    call()
    torch.cuda.synchronize()
    for cap in (5, 2):
        dg.dg_set_num_sms(cap)
        try:
            for _ in range(5):
                grids = _grids(call, tmp_path)
                if grids:                                # (a process's first profiles can be empty)
                    break
        finally:
            dg.dg_set_num_sms(0)
        if not grids:
            pytest.skip("the profiler records no kernels here")
        assert max(grids) <= cap, f"grids {grids} with a cap of {cap} SMs"
