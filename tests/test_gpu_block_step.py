"""The operators as a decoding step uses them: the norm's FP8 output into the experts' layer, the router's choices between them, the
layer's output back into the stream. Eager, captured and in every launch mode; against 64 bits; and their grids under dg_set_num_sms."""
import json

import pytest
import torch

import _block_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
T, K, I, E, k = 7, 512, 256, 12, 3
EPS = 1e-6


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield m
    m.dg_set_num_sms(0)
    assert m.dg_get_device_status() == 0


class Step:
    """Weights, inputs and buffers of one layer; `form`: how the weights and the activations' scales are stored."""

    def __init__(self, dg, form, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        e = lambda dt, *s: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        self.dg, self.form = dg, form
        ue = form == "ue8m0"
        self.x, self.attn = (2 * r(T, K)).to(BF), r(T, K).to(BF)
        self.w_post, self.w_pre, self.w_out, self.scale = 1 + 0.2 * r(K), 1 + 0.2 * r(K), 1 + 0.2 * r(K), 0.3 * r(K)
        self.router, self.bias = (r(E, K) * K ** -0.5).to(BF), 0.05 * r(E)
        st = torch.int32 if ue else F32
        if form == "mxfp4":
            q = lambda N, D: (torch.randint(0, 256, (E, N, D // 2), generator=g, device="cuda", dtype=torch.uint8),  # noqa: E731
                              torch.randint(118, 122, (E, N, D // 32), generator=g, device="cuda", dtype=torch.uint8))
        else:
            def q(N, D):
                codes = e(torch.float8_e4m3fn, E, N, D)
                scales = e(st, E, N // 128, -(-D // 512) if ue else D // 128)
                (dg.dg_cast_fp8_ue8m0 if ue else dg.dg_cast_fp8)((r(E, N, D) * D ** -0.5).to(BF), Xb=codes, sB=scales)
                return codes.view(torch.uint8), scales
        self.w1, self.s1 = q(2 * I, K)
        self.w2, self.s2 = q(K, I)
        self.h, self.y = e(BF, T, K), e(BF, T, K)
        self.q, self.sq = e(torch.uint8, T, K), e(st, -(-K // 512) if ue else K // 128, 8)
        self.yb, self.ids, self.weights = e(BF, T, K), e(torch.int32, T, k), e(F32, T, k)
        self.out, self.next = e(BF, T, K), e(BF, T, K)
        self.logits = e(F32, T, E)

    def run(self):
        dg, ue = self.dg, self.form == "ue8m0"
        norm = dg.dg_residual_norm_ue8m0 if ue else dg.dg_residual_norm
        norm(self.x, self.w_pre, B=self.attn, w_after=self.w_post, scale=self.scale, R=self.h, Y=self.yb, Yq=self.q, sY=self.sq, eps=EPS)
        self.logits.copy_(self.yb.float() @ self.router.float().t())
        dg.dg_route_topk(self.logits, self.ids, self.weights, bias=self.bias, score="sigmoid", factor=2.0)
        moe = {"": dg.dg_fp8_moe_swiglu, "ue8m0": dg.dg_fp8_moe_swiglu_ue8m0, "mxfp4": dg.dg_fp8_moe_swiglu_mxfp4}[self.form]
        moe(self.q, self.sq, self.w1, self.s1, self.w2, self.s2, self.ids, self.weights, self.y)
        dg.dg_residual_norm(self.h, self.w_out, B=self.y, R=self.out, Y=self.next, eps=EPS)

    def outputs(self):
        torch.cuda.synchronize()
        return {n: getattr(self, n).clone() for n in ("h", "yb", "q", "sq", "ids", "weights", "y", "out", "next")}


@pytest.mark.parametrize("form", ["", "ue8m0", "mxfp4"])
def test_step_against_the_definitions(dg, form):
    """Each operator's output against the definition on the outputs of the one before it, which the others read."""
    s = Step(dg, form)
    s.run()
    o = s.outputs()
    want = R.norm(s.x, s.w_pre, s.attn, s.w_post, None, s.scale, EPS, BF)
    R.close(o["h"], want["R"], "stream")
    R.close(o["yb"], want["Y"], "norm")
    rows = R.rows_value(o["q"], o["sq"], form == "ue8m0")
    codes, _ = R.cast_rows(*want["y"], form == "ue8m0")
    R.close(rows, codes, "norm in FP8")
    ids, w = R.route(s.logits, s.bias, k, "sigmoid", True, 2.0)
    assert torch.equal(o["ids"].cpu(), ids) and torch.allclose(o["weights"].cpu().double(), w, rtol=2.0 ** -17, atol=0)
    R.close(o["y"], R.moe(o["q"], o["sq"], s.w1, s.s1, s.w2, s.s2, o["ids"], o["weights"], form, BF), "experts")
    want = R.norm(o["h"], s.w_out, o["y"], None, None, None, EPS, BF)
    R.close(o["out"], want["R"], "next stream")
    R.close(o["next"], want["Y"], "next norm")


@pytest.mark.parametrize("form", ["", "ue8m0", "mxfp4"])
def test_step_in_every_launch_mode_eager_and_captured(dg, form):
    s = Step(dg, form)
    s.run()
    want = s.outputs()
    before = dg.dg_get_pdl()
    try:
        for pdl in (True, False, None):
            dg.dg_set_pdl(pdl)
            for _ in range(3):
                s.y.fill_(7)
                s.run()
            got = s.outputs()
            assert all(torch.equal(want[n], got[n]) for n in want), pdl
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                s.run()
                s.run()
            for n in ("h", "q", "ids", "y", "out"):
                getattr(s, n).zero_()
            g.replay()
            g.replay()
            got = s.outputs()
            assert all(torch.equal(want[n], got[n]) for n in want), (pdl, "captured")
    finally:
        dg.dg_set_pdl(before)


def test_new_values_reach_every_operator_of_a_captured_step(dg):
    s, other = Step(dg, ""), Step(dg, "", seed=1)
    s.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    other.run()
    want = other.outputs()
    for n in ("x", "attn", "w_post", "w_pre", "w_out", "scale", "router", "bias", "w1", "s1", "w2", "s2"):
        getattr(s, n).copy_(getattr(other, n))
    g.replay()
    got = s.outputs()
    assert all(torch.equal(want[n], got[n]) for n in want)


def _grids(run, path):
    """(kernel, CTAs) of the library's launches; a process's first profiles can be empty."""
    run()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
            run()
            torch.cuda.synchronize()
        p.export_chrome_trace(str(path))
        events = json.loads(path.read_text())["traceEvents"]
        found = [(e["name"][:60], e["args"]["grid"]) for e in events if e.get("cat") == "kernel" and "dg::" in e["name"]]
        if found:
            return [(n, g[0] * g[1] * g[2]) for n, g in found]
    pytest.skip("the profiler records no kernels here")


def test_no_launch_has_more_ctas_than_the_cap(dg, tmp_path):
    s = Step(dg, "")
    M = 300
    x, w = torch.randn(M, K, device="cuda").to(BF), torch.ones(K, device="cuda")
    rstd, dx, dw = torch.ones(M, device="cuda"), torch.empty(M, K, device="cuda", dtype=BF), torch.empty(K, device="cuda")
    b4, s4 = torch.zeros(4096, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(4096, K // 32, dtype=torch.uint8, device="cuda")
    d = torch.empty(T, 4096, device="cuda", dtype=BF)
    sq = torch.ones(K // 128, 8, device="cuda")
    l, ids, wt = torch.randn(M, 40, device="cuda"), torch.empty(M, 4, dtype=torch.int32, device="cuda"), torch.empty(M, 4, device="cuda")

    def run():
        s.run()
        dg.dg_residual_norm_backward(x, x, rstd, w, dX=dx, dW=dw)
        dg.dg_route_topk(l, ids, wt)
        dg.dg_route_topk_backward(wt, l, ids, l.clone())
        dg.dg_fp8_mxfp4_gemm_nt(s.q, sq, b4, s4, d)

    for cap in (1, 3):
        dg.dg_set_num_sms(cap)
        found = _grids(run, tmp_path / "trace.json")
        assert len(found) >= 11 and all(n <= cap for _, n in found), found
    dg.dg_set_num_sms(0)
    assert max(n for _, n in _grids(run, tmp_path / "trace.json")) > 3
