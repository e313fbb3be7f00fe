"""The gated projection in the dense and contiguous forms, its backward pass, and the contiguous product with
B stored [G, K, N], for FP32 and packed UE8M0 scales, against plain implementations in 64 bits.

Tolerances. A product's FP32 value may be off by (K + 8) roundings of 2^-24 of S, the sum of the magnitudes
of its terms; a stored BF16 value by 2^-8 of itself more. H = silu(g)·u passes the errors of g and u on
through its derivatives (|silu'| <= 1.1) and adds the fast exponential's and division's, 1e-5 of |H|. An
E4M3 code is within half a step of what it stands for: 2^-4 of it, or 2^-10 of its scale near zero.
"""
import numpy as np
import pytest
import torch

import _train_ref as R

pytestmark = pytest.mark.gpu

SCALES = ["fp32", "ue8m0"]
SEED, OFFSET = 1234567890123456789, 42


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    assert m.dg_get_device_status() == 0
    yield m
    m.dg_set_wait_limit_us(-1)
    assert m.dg_get_device_status() == 0


def _fn(dg, name, scales, f32=False):
    return getattr(dg, name + ("_ue8m0" if scales == "ue8m0" else "") + ("_f32" if f32 else ""))


def _operand(rng, M, N, gr, gc, scales, size=1.0):
    """A random [M, N] operand with gr x gc scale groups: (codes, scales [.., ..], its values in 64 bits)."""
    x = (rng.standard_normal((M, N)) * np.exp(rng.uniform(-1.5, 1.5, (M, 1))) * size).astype(np.float32)
    q, s = R.cast_groups(x, gr, gc, scales == "ue8m0")
    s64 = np.ldexp(1.0, s.astype(np.int64) - 127) if scales == "ue8m0" else s.astype(np.float64)
    return q, s, R.e4m3_values(q) * R.spread(s64, gr, gc, M, N)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _ue(scales):
    return scales == "ue8m0"


def _d64(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _product(x, w):
    """x @ w.T in 64 bits and the sum of magnitudes, on the GPU's FP64 units."""
    x, w = _d64(x), _d64(w)
    return (x @ w.T).cpu().numpy(), (x.abs() @ w.abs().T).cpu().numpy()


class Problem:
    """A dense (G = None) or contiguous problem: operands on the device, pre-activations in 64 bits."""

    def __init__(self, M, I, K, scales, sizes=None, seed=0, holes=()):
        rng = np.random.default_rng(seed)
        self.scales, self.I, self.K = scales, I, K
        G = 1 if sizes is None else len(sizes)
        if sizes is None:
            self.M, self.index = M, None
            spans = [(0, M)]
        else:
            spans, at = [], 0
            for n in sizes:
                spans.append((at, at + n))
                at += 128 * R.cdiv(n, 128)
            self.M = at + 128                                   # an unused block at the end
            self.index = np.full(self.M, -1, np.int32)
            for g, (a, b) in enumerate(spans):
                self.index[a:b] = g
            for h in holes:                                     # padding inside a group
                self.index[h] = -1
        q, s, x64 = _operand(rng, self.M, K, 1, 128, scales)
        self.A, self.sA = _dev(q), _dev(R.lay_lines(s, _ue(scales)))
        Bs = [_operand(rng, 2 * I, K, 128, 128, scales, 1 / np.sqrt(K)) for _ in range(G)]
        B, sB = np.stack([b[0] for b in Bs]), np.stack([R.lay_last(b[1], _ue(scales)) for b in Bs])
        self.B, self.sB = (_dev(B[0]), _dev(sB[0])) if sizes is None else (_dev(B), _dev(sB))
        self.d, self.size = np.zeros((self.M, 2 * I)), np.zeros((self.M, 2 * I))
        for g, (a, b) in enumerate(spans):
            self.d[a:b], self.size[a:b] = _product(x64[a:b], Bs[g][2])
        self.live = np.ones(self.M, bool) if sizes is None else self.index >= 0
        self.m_indices = None if sizes is None else _dev(self.index)

    def run(self, dg, f32, save=True, p=0.0, rng=None):
        H = torch.full((self.M, self.I), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        GU = torch.full((self.M, 2 * self.I), float("nan"), dtype=torch.bfloat16, device="cuda") if save else None
        if self.index is None:
            _fn(dg, "dg_fp8_gemm_nt_swiglu", self.scales, f32)(self.A, self.sA, self.B, self.sB, H, GU=GU, rng=rng, p=p)
        else:
            _fn(dg, "dg_fp8_grouped_contiguous_swiglu", self.scales, f32)(self.A, self.sA, self.B, self.sB, self.m_indices,
                                                                          H, GU=GU, rng=rng, p=p)
        torch.cuda.synchronize()
        return H, GU

    def check(self, dg, p=0.0):
        rng = R.rng_tensor(SEED, OFFSET) if p > 0 else None
        H32, GU = self.run(dg, True, p=p, rng=rng)
        H, GU2 = self.run(dg, False, p=p, rng=rng)
        Hn, _ = self.run(dg, False, save=False, p=p, rng=rng)
        live = torch.from_numpy(self.live).cuda()             # (the sentinels' NaN bits differ by type)
        assert torch.equal(H[live].view(torch.int16), H32[live].to(torch.bfloat16).view(torch.int16)), "BF16 H is not FP32 H rounded"
        assert torch.equal(GU.view(torch.int16), GU2.view(torch.int16))
        assert torch.equal(H.view(torch.int16), Hn.view(torch.int16)), "saving GU changed H"
        h, gu = H32.double().cpu().numpy(), GU.double().cpu().numpy()
        assert np.isnan(h[~self.live]).all() and np.isnan(gu[~self.live]).all(), "padding rows were written"
        h, gu, d = h[self.live], gu[self.live], self.d[self.live]
        e = (self.K + 8) * 2.0 ** -24 * self.size[self.live]
        assert (np.abs(gu - d) <= e + 2.0 ** -8 * np.abs(d)).all()
        I = self.I
        g, u, eg, eu = d[:, :I], d[:, I:], e[:, :I], e[:, I:]
        want = R.gate(g, u)
        tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(g) * eu + 1e-5 * np.abs(want)
        if p > 0:
            keep = R.keep_mask(0, self.M * I, p, SEED, OFFSET).reshape(self.M, I)[self.live]
            want, tol = np.where(keep, want * R.keep_scale(p), 0), np.where(keep, tol * R.keep_scale(p) + 1e-6 * np.abs(want), 0)
        assert (np.abs(h - want) <= tol).all()


@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("M,I,K", [(1, 128, 16), (1, 256, 1040), (3, 384, 144), (8, 128, 7168), (9, 256, 528), (16, 128, 80), (17, 128, 144), (64, 128, 640), (127, 128, 128),
                                   (128, 256, 272), (129, 128, 1024), (300, 384, 528), (257, 1024, 2064), (300, 1920, 3600)])   # the last: 128-column tiles, K split
def test_dense(dg, M, I, K, scales):
    Problem(M, I, K, scales).check(dg)


@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("sizes,I,K", [([0, 1, 127, 128], 128, 272), ([130, 0, 64], 256, 144), ([5], 384, 1040),
                                       ([300, 7, 0, 0, 129], 128, 512),
                                       ([700, 0, 1300, 100], 1024, 272), ([140, 0, 40], 1920, 3600)])   # 128-column tiles
def test_contiguous(dg, sizes, I, K, scales):
    Problem(None, I, K, scales, sizes=sizes, holes=[2] if sizes[0] > 4 else []).check(dg)


@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout_in_the_epilogue(dg, scales, p):
    Problem(5, 256, 1040, scales).check(dg, p)            # few tokens: no tiles
    Problem(13, 128, 2064, scales).check(dg, p)
    Problem(40, 256, 1040, scales).check(dg, p)           # K split in a cluster
    Problem(300, 128, 272, scales).check(dg, p)
    Problem(None, 128, 272, scales, sizes=[100, 0, 200], holes=[50]).check(dg, p)
    Problem(None, 1024, 272, scales, sizes=[700, 0, 1300, 100], holes=[50]).check(dg, p)
    Problem(300, 1920, 3600, scales).check(dg, p)


@pytest.mark.parametrize("scales", SCALES)
def test_split_paths_agree(dg, scales):
    """K split in clusters and through the workspace: the same partials in the same order, the same bits."""
    for prob in (Problem(20, 256, 2048, scales), Problem(None, 128, 2048, scales, sizes=[30, 0, 100], holes=[3])):
        on = prob.run(dg, True)
        prev = dg.dg_set_cluster_split(False)
        try:
            off = prob.run(dg, True)
            prob.check(dg, 0.1)
        finally:
            dg.dg_set_cluster_split(prev)
        for a, b in zip(on, off):
            assert torch.equal(a.view(torch.int8), b.view(torch.int8))


@pytest.mark.parametrize("scales", SCALES)
def test_tail_split(dg, scales):
    prob = Problem(1280, 2048, 2048, scales)              # 160 tiles: 8 past one wave of 152
    prob.check(dg, 0.1)
    prev = dg.dg_set_tail_splits(1)
    try:
        prob.check(dg)
    finally:
        dg.dg_set_tail_splits(prev)


@pytest.mark.parametrize("scales", SCALES)
def test_bad_group_index_is_flagged(dg, scales):
    prob = Problem(None, 128, 256, scales, sizes=[100, 60])
    ok, _ = prob.run(dg, False)
    prob.m_indices[7] = 9
    H, GU = prob.run(dg, False)
    assert dg.dg_get_device_status() & dg.DG_DEV_BAD_GROUP_INDEX
    assert torch.isnan(H[7]).all() and torch.isnan(GU[7]).all()
    rest = torch.arange(prob.M, device="cuda") != 7
    assert torch.equal(H[rest].view(torch.int16), ok[rest].view(torch.int16))


@pytest.mark.parametrize("scales", SCALES)
def test_timeout_and_recovery(dg, scales):
    for prob in (Problem(300, 256, 1024, scales), Problem(300, 1920, 3600, scales), Problem(1280, 2048, 272, scales),
                 Problem(20, 256, 2048, scales), Problem(None, 128, 256, scales, sizes=[100, 60])):
        ref, _ = prob.run(dg, False)
        prev = dg.dg_set_wait_limit_us(0)
        try:
            prob.run(dg, False)
            status = dg.dg_get_device_status()
        finally:
            dg.dg_set_wait_limit_us(prev)
        assert status & dg.DG_DEV_TIMEOUT
        again, _ = prob.run(dg, False)
        assert dg.dg_get_device_status() == 0
        assert torch.equal(again.view(torch.int16), ref.view(torch.int16))


def test_forward_refusals(dg):
    p = Problem(16, 128, 256, "fp32")
    H = torch.empty(16, 128, dtype=torch.bfloat16, device="cuda")
    call = dg.dg_fp8_gemm_nt_swiglu
    with pytest.raises(dg.DGError):
        call(p.A, p.sA, p.B, p.sB, H, p=0.1)                              # no rng
    with pytest.raises(dg.DGError):
        call(p.A, p.sA, p.B, p.sB, H, rng=R.rng_tensor(1, 1), p=1.0)
    with pytest.raises(ValueError):
        call(p.A, p.sA, p.B, p.sB, H, GU=torch.empty(16, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        call(p.A, p.sA, p.B, p.sB, torch.empty(16, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        call(p.A, p.sA, p.B, p.sB, H.float())
    with pytest.raises(TypeError):
        call(p.A, p.sA, p.B, p.sB, H, rng=torch.zeros(2, device="cuda"), p=0.1)
    with pytest.raises(dg.DGError) as e:                                  # 2I = 192
        call(p.A, p.sA, p.B[:192], p.sB, H[:, :96].contiguous())
    assert e.value.status == dg.DG_ERR_ALIGNMENT
    call(p.A[:0], p.sA[:, :0], p.B, p.sB, H[:0])                          # no tokens: nothing to do


# ------------------------------------------------------------------------------------- backward

class Backward:
    def __init__(self, M, I, scales, seed=0, pad=(), p=0.0):
        rng = np.random.default_rng(seed)
        self.M, self.I, self.scales, self.p = M, I, scales, p
        gu = R.bf16(rng.standard_normal((M, 2 * I)) * 3)
        dh = R.bf16(rng.standard_normal((M, I)) * 0.01 * np.exp(rng.uniform(-4, 4, (M, 1))))
        gu[0, :2], dh[0, 1] = (60.0, -90.0), 1.0                        # the gate saturated on both sides
        self.m_indices = None
        live = np.ones(M, bool)
        if len(pad):
            live[list(pad)] = False
            idx = np.where(live, 0, -1).astype(np.int32)
            self.m_indices = _dev(idx)
        self.live = live
        self.GU, self.dH = R.to_dev_bf16(gu), R.to_dev_bf16(dh)
        if len(pad):
            self.GU[~torch.from_numpy(live).cuda()] = float("nan")       # what no one wrote
            self.dH[~torch.from_numpy(live).cuda()] = float("nan")
        t = dh.astype(np.float64)
        keep = R.keep_mask(0, M * I, p, SEED, OFFSET).reshape(M, I) if p > 0 else np.ones((M, I), bool)
        q = R.keep_scale(p)
        t = np.where(keep, t * q, 0)
        g, u = gu[:, :I].astype(np.float64), gu[:, I:].astype(np.float64)
        dg, du = R.gate_grad(g, u, t)
        self.d = np.where(live[:, None], np.concatenate([dg, du], 1), 0)
        self.h = np.where(live[:, None] & keep, R.gate(g, u) * q, 0)
        # the terms that cancel in 1 + g(1 - s): the error of dg is of their size
        self.size = np.where(live[:, None], np.concatenate([np.abs(t * u) * (1 + np.abs(g)), np.abs(du)], 1), 0)

    def run(self, dg, rows=True, cols=True, blocks=True):
        ue, M, I = _ue(self.scales), self.M, self.I
        sdt = torch.int32 if ue else torch.float32
        w = (lambda n: R.cdiv(n, 4)) if ue else (lambda n: n)
        code = lambda n: torch.full((M, n), 0x55, dtype=torch.uint8, device="cuda")      # noqa: E731
        sc = lambda *s: torch.full(s, 0x55555555, dtype=torch.int32, device="cuda").view(sdt)  # noqa: E731
        mb, nb = R.cdiv(M, 128), 2 * I // 128
        out = {}
        if rows:
            out.update(dGUr=code(2 * I), sR=sc(w(nb), 4 * R.cdiv(M, 4)))
        if cols:
            out.update(dGUc=code(2 * I), sC=sc(w(mb), 2 * I))
        if blocks:
            out.update(Hb=code(I), sHb=sc(I // 128, w(mb)))
        _fn(dg, "dg_swiglu_backward_fp8", self.scales)(
            self.dH, self.GU, m_indices=self.m_indices, rng=R.rng_tensor(SEED, OFFSET) if self.p > 0 else None, p=self.p, **out)
        torch.cuda.synchronize()
        return out

    def close(self, q, s, want, size, gr, gc):
        """Codes q with scales s (at every group) against `want`: half a step, the FP32 error, and the scale."""
        err32 = 2e-6 * size + 1e-5 * np.abs(want)
        step = np.maximum(2.0 ** -4 * (np.abs(want) + err32), 2.0 ** -10 * s)
        assert (np.abs(R.e4m3_values(q) * s - want) <= step * 1.0001 + err32).all()
        M, N = want.shape
        pad = np.zeros((gr * R.cdiv(M, gr), gc * R.cdiv(N, gc)))
        pad[:M, :N] = np.abs(want)
        slack = np.zeros_like(pad)
        slack[:M, :N] = err32
        group = lambda x: x.reshape(R.cdiv(M, gr), gr, R.cdiv(N, gc), gc).max(axis=(1, 3))  # noqa: E731
        top, off = group(pad), group(slack)
        s = s[::gr, ::gc]
        none = top == 0
        assert (s[none] == 1).all()
        lo, hi = (top - off) / 448 * (1 - 1e-6), (top + off) / 448 * (2 if _ue(self.scales) else 1) * (1 + 1e-6)
        assert ((s >= lo) & (s <= hi))[~none].all()

    def check(self, dg):
        out, M, I = self.run(dg), self.M, self.I
        nb, mb = 2 * I // 128, R.cdiv(M, 128)
        self.close(out["dGUr"], R.spread(R.unlay_lines(out["sR"], M, nb), 1, 128, M, 2 * I), self.d, self.size, 1, 128)
        self.close(out["dGUc"], R.spread(R.unlay_lines(out["sC"], 2 * I, mb).T, 128, 1, M, 2 * I), self.d, self.size, 128, 1)
        self.close(out["Hb"], R.spread(R.unlay_last(out["sHb"], mb).T, 128, 128, M, I), self.h, np.abs(self.h), 128, 128)
        ld = out["sR"].shape[1]
        if ld > M:                                                      # the filler past the rows
            assert (out["sR"][:, M:] == (0x7F7F7F7F if _ue(self.scales) else 0)).all()
        for part in (dict(cols=False, blocks=False), dict(rows=False, blocks=False), dict(rows=False), dict(cols=False)):
            for k, v in self.run(dg, **part).items():
                assert torch.equal(v.view(torch.int8), out[k].view(torch.int8)), f"{k} differs when asked for with {part}"
        return out


@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("M,I", [(1, 128), (3, 256), (127, 128), (128, 128), (130, 384), (333, 128), (700, 640)])
def test_backward_forms(dg, M, I, scales):
    Backward(M, I, scales).check(dg)


@pytest.mark.parametrize("scales", SCALES)
def test_backward_dropout_and_padding(dg, scales):
    Backward(200, 256, scales, p=0.3).check(dg)
    Backward(384, 128, scales, p=0.1, pad=list(range(100, 128)) + list(range(256, 384))).check(dg)


@pytest.mark.parametrize("scales", SCALES)
def test_backward_against_differences(dg, scales):
    """The dequantised gradients against central differences of sum(dH·H) in 64 bits (truncation e²/6·|h'''|,
    |h'''| <= |u|): half an E4M3 step."""
    b = Backward(130, 128, scales)
    out = b.run(dg, cols=False, blocks=False)
    g, u = (x.double().cpu().numpy() for x in (b.GU[:, :128], b.GU[:, 128:]))
    t, e = b.dH.double().cpu().numpy(), 1e-4
    num = np.concatenate([t * (R.gate(g + e, u) - R.gate(g - e, u)) / (2 * e),
                          t * (R.gate(g, u + e) - R.gate(g, u - e)) / (2 * e)], 1)
    s = R.spread(R.unlay_lines(out["sR"], 130, 2), 1, 128, 130, 256)
    slack = 1e-7 * np.abs(np.concatenate([t, t], 1)) * (1 + np.abs(np.concatenate([u * (1 + np.abs(g)), g], 1))) + 1e-5 * np.abs(num)
    assert (np.abs(R.e4m3_values(out["dGUr"]) * s - num) <= np.maximum(2.0 ** -4 * np.abs(num), 2.0 ** -10 * s) * 1.0001 + 20 * slack).all()


def test_backward_refusals(dg):
    b = Backward(16, 128, "fp32")
    q, s = torch.empty(16, 256, dtype=torch.uint8, device="cuda"), torch.empty(2, 16, device="cuda")
    with pytest.raises(dg.DGError):
        dg.dg_swiglu_backward_fp8(b.dH, b.GU)                            # no form of the gradients
    with pytest.raises(dg.DGError):
        dg.dg_swiglu_backward_fp8(b.dH, b.GU, dGUr=q)                    # codes without scales
    with pytest.raises(ValueError):
        dg.dg_swiglu_backward_fp8(b.dH, b.GU[:, :128].contiguous(), dGUr=q, sR=s)
    with pytest.raises(ValueError):
        dg.dg_swiglu_backward_fp8(b.dH, b.GU, dGUr=q, sR=s[:1])
    with pytest.raises(TypeError):
        dg.dg_swiglu_backward_fp8(b.dH.float(), b.GU, dGUr=q, sR=s)
    with pytest.raises(dg.DGError):
        dg.dg_swiglu_backward_fp8(b.dH, b.GU, dGUr=q, sR=s, p=0.5)       # no rng
    with pytest.raises(dg.DGError) as e:                                 # I = 96
        dg.dg_swiglu_backward_fp8(b.dH[:, :96].contiguous(), b.GU[:, :192].contiguous(), dGUr=q[:, :192].contiguous(), sR=s)
    assert e.value.status == dg.DG_ERR_ALIGNMENT
    dg.dg_swiglu_backward_fp8(b.dH[:0], b.GU[:0], dGUr=q[:0], sR=s[:, :0])


# ------------------------------------------------------------------------------------- contiguous NN

@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("sizes,N,K", [([0, 1, 127, 128], 16, 128), ([130, 0, 64], 272, 256), ([5], 144, 2048), ([300, 7, 129], 528, 384)])
def test_contiguous_nn(dg, sizes, N, K, scales):
    rng = np.random.default_rng(3)
    G = len(sizes)
    spans, at = [], 0
    for n in sizes:
        spans.append((at, at + n))
        at += 128 * R.cdiv(n, 128)
    M = at + 128
    index = np.full(M, -1, np.int32)
    for g, (a, b) in enumerate(spans):
        index[a:b] = g
    q, s, x64 = _operand(rng, M, K, 1, 128, scales)
    Ws = [_operand(rng, K, N, 128, 128, scales) for _ in range(G)]
    B = _dev(np.stack([w[0] for w in Ws]))
    sB = _dev(np.stack([R.lay_last(np.ascontiguousarray(w[1].T), _ue(scales)) for w in Ws]))
    A, sA, idx = _dev(q), _dev(R.lay_lines(s, _ue(scales))), _dev(index)
    D32 = torch.full((M, N), float("nan"), device="cuda")
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    _fn(dg, "dg_fp8_grouped_contiguous_nn", scales, True)(A, sA, B, sB, idx, D32)
    _fn(dg, "dg_fp8_grouped_contiguous_nn", scales)(A, sA, B, sB, idx, D)
    live = idx >= 0                                                    # (the sentinels' NaN bits differ by type)
    assert torch.equal(D[live].view(torch.int16), D32[live].to(torch.bfloat16).view(torch.int16))
    assert torch.isnan(D[~live]).all()
    d = D32.double().cpu().numpy()
    assert np.isnan(d[index < 0]).all()
    for g, (a, b) in enumerate(spans):
        ref, size = _product(x64[a:b], Ws[g][2].T)
        assert (np.abs(d[a:b] - ref) <= (K + 8) * 2.0 ** -24 * size).all()
    # the NT call on the transposed weights: the same products in the same order
    Dt = torch.full((M, N), float("nan"), device="cuda")
    sBt = _dev(np.stack([R.lay_last(np.ascontiguousarray(w[1].T), _ue(scales)) for w in Ws]))
    _fn(dg, "dg_fp8_grouped_contiguous", scales, True)(A, sA, B.transpose(1, 2).contiguous(), sBt, idx, Dt)
    assert torch.equal(Dt.view(torch.int32), D32.view(torch.int32))


def test_contiguous_nn_refusals(dg):
    M, N, K, G = 128, 64, 256, 2
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")   # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")                        # noqa: E731
    idx = torch.zeros(M, dtype=torch.int32, device="cuda")
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    call = dg.dg_fp8_grouped_contiguous_nn
    with pytest.raises(dg.DGError) as e:                               # K not whole blocks
        call(u8(M, 192), f(2, M), u8(G, 192, N), f(G, 1, 2), idx, D)
    assert e.value.status == dg.DG_ERR_ALIGNMENT
    with pytest.raises(dg.DGError):                                    # N % 16
        call(u8(M, K), f(2, M), u8(G, K, 72), f(G, 1, 2), idx, torch.empty(M, 72, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        call(u8(M, K), f(2, M), u8(G, N, K), f(G, 1, 2), idx, D)       # the NT layout
    with pytest.raises(ValueError):
        call(u8(M, K), f(2, M), u8(G, K, N), f(G, 2, 1), idx, D)


# ------------------------------------------------------------------------------------- the whole step

@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("grouped", [False, True])
def test_training_chain(dg, scales, grouped):
    """dX and dW from the kernel's own codes within the products' bounds, the same with programmatic
    dependent launch, and from a captured graph."""
    I, K, p = 256, 272, 0.1
    rng = np.random.default_rng(8)
    sizes = [100, 0, 130] if grouped else [150]
    starts = np.concatenate([[0], np.cumsum([128 * R.cdiv(n, 128) if grouped else n for n in sizes])])
    M, G = int(starts[-1]), len(sizes)
    live = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, sizes)]).astype(int)
    b = Backward(M, I, scales, p=p, pad=sorted(set(range(M)) - set(live.tolist())))
    if grouped:
        index = np.full(M, -1, np.int32)
        for g, n in enumerate(sizes):
            index[starts[g]:starts[g] + n] = g
        b.m_indices = _dev(index)
    ws = [_operand(rng, 2 * I, K, 128, 128, scales) for _ in range(G)]
    W, sWt = np.stack([w[0] for w in ws]), np.stack([R.lay_last(np.ascontiguousarray(w[1].T), _ue(scales)) for w in ws])
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[sorted(set(range(M)) - set(live.tolist()))] = 0
    xq, xs = R.cast_groups(x, 128, 128, _ue(scales))
    xs64 = np.ldexp(1.0, xs.astype(np.int64) - 127) if _ue(scales) else xs.astype(np.float64)
    x64 = R.e4m3_values(xq) * R.spread(xs64, 128, 128, M, K)
    W, sWt, Xb, sXb = _dev(W), _dev(sWt), _dev(xq), _dev(R.lay_last(np.ascontiguousarray(xs.T), _ue(scales)))
    offsets = _dev(starts.astype(np.int32))
    dX, dW = torch.zeros(M, K, device="cuda"), torch.zeros(G, 2 * I, K, device="cuda")
    got = {}

    def step():
        got.update(b.run(dg) if not torch.cuda.is_current_stream_capturing() else _captured(dg, b, got))
        if grouped:
            _fn(dg, "dg_fp8_grouped_contiguous_nn", scales, True)(got["dGUr"], got["sR"], W, sWt, b.m_indices, dX)
            _fn(dg, "dg_fp8_k_grouped_gemm_tn_contiguous", scales, True)(got["dGUc"], got["sC"], Xb, sXb, offsets, dW)
        else:
            _fn(dg, "dg_fp8_gemm_nn", scales, True)(got["dGUr"], got["sR"], W[0], sWt[0], dX, M, K, 2 * I)
            _fn(dg, "dg_fp8_gemm_tn", scales, True)(got["dGUc"], got["sC"], Xb, sXb, dW[0], 2 * I, K, M)

    step()
    torch.cuda.synchronize()
    nb, mb = 2 * I // 128, R.cdiv(M, 128)
    r64 = R.e4m3_values(got["dGUr"]) * R.spread(R.unlay_lines(got["sR"], M, nb), 1, 128, M, 2 * I)
    c64 = R.e4m3_values(got["dGUc"]) * R.spread(R.unlay_lines(got["sC"], 2 * I, mb).T, 128, 1, M, 2 * I)
    for g, n in enumerate(sizes):
        a, e = int(starts[g]), int(starts[g]) + n
        ref, size = _product(r64[a:e], ws[g][2].T)
        assert (np.abs(dX[a:e].double().cpu().numpy() - ref) <= (2 * I + 8) * 2.0 ** -24 * size).all()
        ref, size = _product(c64[a:e].T, x64[a:e].T)
        assert (np.abs(dW[g].double().cpu().numpy() - ref) <= (n + 8) * 2.0 ** -24 * size).all()
    want = dX.clone(), dW.clone()
    prev = dg.dg_set_pdl(True)
    try:
        for _ in range(3):
            dX.fill_(0), dW.fill_(0)
            step()
    finally:
        dg.dg_set_pdl(prev)
    torch.cuda.synchronize()
    assert torch.equal(dX, want[0]) and torch.equal(dW, want[1])
    graph = torch.cuda.CUDAGraph()
    b.rng = R.rng_tensor(SEED, OFFSET)
    with torch.cuda.graph(graph):
        step()
    dX.fill_(0), dW.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dX, want[0]) and torch.equal(dW, want[1])


def _captured(dg, b, out):
    _fn(dg, "dg_swiglu_backward_fp8", b.scales)(b.dH, b.GU, m_indices=b.m_indices, rng=b.rng, p=b.p, **out)
    return out


def test_the_binding_s_two_paths_make_the_same_call(dg, monkeypatch):
    """Arguments checked by the compiled short path and by Python: the same bits."""
    prob, back = Problem(200, 128, 272, "fp32"), Backward(200, 128, "ue8m0", p=0.1)
    x = torch.randn(200, 144, device="cuda").bfloat16()
    rng = R.rng_tensor(SEED, OFFSET)

    def calls():
        out = list(prob.run(dg, False, p=0.1, rng=rng)) + list(back.run(dg).values())
        q, s, y = torch.zeros(200, 144, dtype=torch.uint8, device="cuda"), torch.zeros(2, 200, device="cuda"), torch.empty_like(x)
        dg.dg_cast_fp8(x, Xr=q, sR=s)
        dg.dg_dropout(x, y, rng, 0.25, R=x)
        d = torch.empty(200, 256, dtype=torch.bfloat16, device="cuda")
        dg.dg_fp8_gemm_nt(prob.A, prob.sA, prob.B, prob.sB, d)
        return out + [q, s, y, d]

    first = calls()
    assert dg._bind() is not dg._NoBind, "the short path is not built"
    monkeypatch.setattr(dg, "_bind", lambda: dg._NoBind)
    for a, b in zip(first, calls()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
