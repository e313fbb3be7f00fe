"""Early start always, never and where it pays (the default): the same bits, eager and from a captured graph.

Each chain's kernels read what the one before wrote, with the buffers poisoned first, so that a kernel that read its
inputs too early would be caught. What stands ahead of a call is also a fill, a copy and, in a captured graph, the
join of two streams: launches that may start early have to be right behind any of them.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

MODES = [None, True, False]


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    prev = m.dg_get_pdl()
    yield m
    assert m.dg_get_pdl() is prev, "a test left another launch mode behind"
    assert m.dg_get_device_status() == 0


@pytest.fixture(params=MODES, ids=["short", "always", "never"])
def mode(dg, request):
    prev = dg.dg_set_pdl(request.param)
    yield request.param
    dg.dg_set_pdl(prev)


def _cdiv(a, b):
    return -(-a // b)


class Step:
    """One expert layer's worth of calls on M rows: casts, gated projection, down projection, dropout, backward, dX, dW."""

    def __init__(self, dg, scales, M=384, K=512, I=256):
        self.dg, self.ue = dg, scales == "ue8m0"
        gen = torch.Generator(device="cuda").manual_seed(5)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
        self.x0, self.dy0, self.w1, self.w2 = r(M, K), r(M, K), r(2 * I, K), r(K, I)
        self.M, self.K, self.I = M, K, I
        self.rng = torch.tensor([11, 3], dtype=torch.int64, device="cuda")
        q = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
        b = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        w = (lambda n: _cdiv(n, 512)) if self.ue else (lambda n: _cdiv(n, 128))
        s = lambda *n: torch.empty(n, dtype=torch.int32 if self.ue else torch.float32, device="cuda")  # noqa: E731
        self.buf = dict(x=b(M, K), dy=b(M, K), xr=q(M, K), sxr=s(w(K), M), xb=q(M, K), sxb=s(K // 128, w(M)), w1q=q(2 * I, K),
                        s1=s(2 * I // 128, w(K)), s1t=s(K // 128, w(2 * I)), w2q=q(K, I), s2=s(K // 128, w(I)), h=b(M, I), gu=b(M, 2 * I),
                        hr=q(M, I), shr=s(w(I), M), y=b(M, K), out=b(M, K), dh=b(M, I), gr=q(M, 2 * I), sgr=s(w(2 * I), M),
                        gc=q(M, 2 * I), sgc=s(w(M), 2 * I), dx=b(M, K), dw=b(2 * I, K), small=b(64, 2112))
        self.dh0 = r(M, I)
        self.a, self.sa = (torch.rand(64, 7168, generator=gen, device="cuda") - 0.5).to(torch.float8_e4m3fn), s(w(7168), 64)
        self.b, self.sb = (torch.rand(2112, 7168, generator=gen, device="cuda") - 0.5).to(torch.float8_e4m3fn), s(17, w(7168))
        for t in (self.sa, self.sb):
            t.fill_(0x7F7E7F7E if self.ue else 0.75)

    def _fn(self, name):
        return getattr(self.dg, name + ("_ue8m0" if self.ue else ""))

    def poison(self):
        for t in self.buf.values():
            t.view(torch.uint8).fill_(0xFF)

    def run(self):
        d, t, cast = self.dg, self.buf, self._fn("dg_cast_fp8")
        t["x"].copy_(self.x0)
        cast(t["x"], Xr=t["xr"], sR=t["sxr"], Xb=t["xb"], sBt=t["sxb"])                 # behind a copy
        cast(self.w1, Xb=t["w1q"], sB=t["s1"], sBt=t["s1t"])
        self._fn("dg_fp8_gemm_nt_swiglu")(t["xr"], t["sxr"], t["w1q"], t["s1"], t["h"], GU=t["gu"], rng=self.rng, p=0.1)
        cast(self.w2, Xb=t["w2q"], sB=t["s2"])
        cast(t["h"], Xr=t["hr"], sR=t["shr"])
        self._fn("dg_fp8_gemm_nt")(t["hr"], t["shr"], t["w2q"], t["s2"], t["y"])
        d.dg_dropout(t["y"], t["out"], self.rng, 0.25, R=t["x"])
        t["small"].zero_()
        self._fn("dg_fp8_gemm_nt")(self.a, self.sa, self.b, self.sb, t["small"])        # split-K, behind a fill
        t["dh"].copy_(self.dh0)
        self._fn("dg_swiglu_backward_fp8")(t["dh"], t["gu"], t["gr"], t["sgr"], t["gc"], t["sgc"], rng=self.rng, p=0.1)
        self._fn("dg_fp8_gemm_nn")(t["gr"], t["sgr"], t["w1q"], t["s1t"], t["dx"], self.M, self.K, 2 * self.I)
        self._fn("dg_fp8_gemm_tn")(t["gc"], t["sgc"], t["xb"], t["sxb"], t["dw"], 2 * self.I, self.K, self.M)

    def outputs(self):
        torch.cuda.synchronize()
        return {k: v.view(torch.uint8).clone() for k, v in self.buf.items()}


def _same(got, want):
    for k in want:
        assert torch.equal(got[k], want[k]), k


def _plain(dg, step):
    prev = dg.dg_set_pdl(False)
    try:
        step.poison()
        step.run()
        out = step.outputs()
    finally:
        dg.dg_set_pdl(prev)
    for k, v in out.items():
        if k in ("h", "gu", "y", "out", "dx", "dw", "small"):
            assert torch.isfinite(v.view(torch.bfloat16).float()).all(), k
    return out


@pytest.mark.parametrize("scales", ["fp32", "ue8m0"])
def test_a_chain_gives_the_same_bits(dg, mode, scales):
    step = Step(dg, scales)
    want = _plain(dg, step)
    for _ in range(10):
        step.poison()
        step.run()
        _same(step.outputs(), want)


@pytest.mark.parametrize("scales", ["fp32", "ue8m0"])
def test_a_captured_chain_gives_the_same_bits(dg, mode, scales):
    step = Step(dg, scales)
    want = _plain(dg, step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.poison()
        step.run()
        step.run()
    for _ in range(5):
        graph.replay()
        _same(step.outputs(), want)


def test_calls_behind_the_join_of_two_streams(dg, mode):
    step = Step(dg, "fp32")
    want = _plain(dg, step)
    t, cast = step.buf, dg.dg_cast_fp8
    side = torch.cuda.Stream()

    def joined():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            t["x"].copy_(step.x0)
            cast(t["x"], Xr=t["xr"], sR=t["sxr"])
        cast(step.w1, Xb=t["w1q"], sB=t["s1"], sBt=t["s1t"])
        torch.cuda.current_stream().wait_stream(side)
        dg.dg_fp8_gemm_nt_swiglu(t["xr"], t["sxr"], t["w1q"], t["s1"], t["h"], GU=t["gu"], rng=step.rng, p=0.1)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.poison()
        joined()
    for _ in range(10):
        graph.replay()
        got = step.outputs()
        assert torch.equal(got["h"], want["h"]) and torch.equal(got["gu"], want["gu"])
    for _ in range(10):
        step.poison()
        joined()
        got = step.outputs()
        assert torch.equal(got["h"], want["h"]) and torch.equal(got["gu"], want["gu"])
