"""The router against the plain 64-bit definition: every id, the weights, the gradient against the formula and against
differences, near ties, masked logits, launch settings and graphs."""
import pytest
import torch

import _block_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield m
    assert m.dg_get_device_status() == 0


def _logits(T, E, dt=F32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (2 * torch.randn(T, E, generator=g, device="cuda")).to(dt), 0.2 * torch.randn(E, generator=g, device="cuda")


def _route(dg, l, k, bias=None, **how):
    T = l.shape[0]
    ids, w = torch.full((T + 1, k), 77, dtype=torch.int32, device="cuda"), torch.full((T + 1, k), 77.0, device="cuda")
    dg.dg_route_topk(l, ids[:T], w[:T], bias=bias, **how)
    assert bool((ids[T] == 77).all()) and bool((w[T] == 77).all())
    return ids[:T], w[:T]


def _check(dg, l, k, bias, score, renorm, factor):
    ids, w = _route(dg, l, k, bias, score=score, renormalize=renorm, factor=factor)
    want_ids, want = R.route(l, bias, k, score, renorm, factor)
    assert torch.equal(ids.cpu(), want_ids)
    # exp (2 ulp), a sum of 32 terms a lane and five levels, a division each: below 2^-17 of the weight
    off = (w.cpu().double() - want).abs()
    assert bool((off <= 2.0 ** -17 * want.abs() + 1e-37).all()), float((off / want.abs().clamp_min(1e-37)).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (5, 33, 33 - 1), (7, 64, 6), (4, 65, 8), (9, 128, 8), (2, 160, 6), (130, 256, 8), (3, 300, 1),
                                   (2, 512, 10), (3, 1000, 32), (2, 1024, 8)])
def test_matches_definition(dg, T, E, k, score, bias, renorm):
    l, b = _logits(T, E)
    _check(dg, l, k, b if bias else None, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bf16_logits_have_many_ties(dg, score):
    l, b = _logits(64, 256, BF)
    _check(dg, l, 8, None, score, True, 1.0)                 # equal logits: the lowest index first
    _check(dg, l, 8, torch.zeros_like(b), score, True, 1.0)
    _check(dg, l, 8, b, score, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_next_to_one_another(dg, score):
    """Keys that FP32 does not tell apart: logits one step apart, scores that saturate, a bias that swallows them."""
    E, k = 96, 12
    l = torch.full((6, E), 1.0, device="cuda")
    step = torch.arange(E, device="cuda", dtype=F32)
    l[0] = 1.0 + step.flip(0) * 2.0 ** -23
    l[1] = 1.0 + step * 2.0 ** -23
    l[2] = 17.0 + step * 0.01                                 # sigmoids round to 1 in FP32
    l[3] = torch.where(step % 2 == 0, 3.0, 3.0 + 2.0 ** -22)
    l[4] = -step * 2.0 ** -20
    l[5] = 1.0
    zero = torch.zeros(E, device="cuda")
    _check(dg, l, k, None, score, False, 1.0)
    _check(dg, l, k, zero, score, False, 1.0)
    _check(dg, l, k, torch.full((E,), 1000.0, device="cuda"), score, False, 1.0)
    _check(dg, l, k, torch.where(step % 3 == 0, 0.5, 0.5 - 2.0 ** -24), score, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_masked_logits(dg, score, bias):
    l, b = _logits(9, 70)
    low = torch.finfo(F32).min
    l[0] = -torch.inf                                        # nothing left
    l[1, 3:] = -torch.inf                                    # fewer than k
    l[2] = low                                               # the type's lowest value is a value
    l[3, ::2] = low
    l[4] = torch.nan
    l[5, 10:20] = torch.nan
    l[6, 5] = 80.0
    l[7, :60] = -torch.inf
    b[40:44] = -torch.inf
    _check(dg, l, 6, b if bias else None, score, False, 1.0)
    _check(dg, l, 6, b if bias else None, score, True, 2.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(12, 12), (13, 12), (40, 31), (40, 32), (32, 32), (33, 32), (256, 8), (300, 32)])
def test_runs_of_near_scores(dg, score, E, k):
    """Pairs, threes and longer runs of logits that share the upper bits of their keys, inside the selection, across its border and
    beyond 32 of them; the same with biases that bring scores of different logits together."""
    g = torch.Generator(device="cuda").manual_seed(E + k)
    T = 48
    l = torch.randn(T, E, generator=g, device="cuda")
    for t in range(T):
        run = (1, 2, 2, 3, 4, 7, 40)[t % 7]
        order = torch.argsort(l[t], descending=True)
        for at in range(t % 5, E - run + 1, run + 1):         # runs one step or none apart, in no order of the indexes
            steps = torch.randint(-1, 2, (run,), generator=g, device="cuda") if t % 2 else torch.arange(run, device="cuda")
            l[t, order[at:at + run]] = l[t, order[at]] * (1 + steps * 2.0 ** -23)
    _check(dg, l, k, None, score, True, 1.0)
    _check(dg, l, k, torch.zeros(E, device="cuda"), score, True, 1.0)
    b = torch.randn(E, generator=g, device="cuda")
    s = R.scores(l[:1], score)[0]
    b = (b[E // 2] + s[E // 2] - s).float()                   # the first token's sums: equal to within a rounding
    _check(dg, l, k, b, score, True, 1.0)


def test_infinite_logits_are_equal(dg):
    l = torch.randn(5, 64, device="cuda")
    l[0, [50, 3, 17]] = torch.inf
    l[1, [7, 8]] = torch.inf
    l[2] = torch.inf
    for k in (2, 8):
        for bias in (None, torch.zeros(64, device="cuda")):
            _check(dg, l, k, bias, "sigmoid", False, 1.0)
    b = torch.zeros(64, device="cuda")
    b[[60, 2, 31]] = torch.inf
    _check(dg, l, 8, b, "sigmoid", False, 1.0)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_zeros_of_both_signs_tie(dg, score, dt):
    """-0 and 0 are the same logit: the lowest index first, with and without a bias."""
    l = torch.zeros(3, 136, device="cuda", dtype=dt)
    l[0, ::2] = -0.0
    l[1, 1::2] = -0.0
    l[2, :70], l[2, 70:] = -0.0, -1.0
    zero = torch.zeros(136, device="cuda")
    for bias in (None, zero, -zero):
        _check(dg, l, 9, bias, score, True, 1.0)


def _gradient(l, ids, dw, score, renorm, factor):
    """From the formulas, in 64 bits, with the sizes of the terms that are added."""
    s = R.scores(l.float(), score)
    ok = ids >= 0
    at = ids.clamp_min(0).long()
    d = torch.where(ok, factor * dw.double(), 0.0)
    ed = d.abs()
    if renorm:
        sel = torch.where(ok, torch.gather(s, 1, at), 0.0)
        total = sel.sum(1, keepdim=True) + 1e-20
        mean = (d * sel).sum(1, keepdim=True) / total
        size = (d.abs() * sel).sum(1, keepdim=True) / total
        d, ed = torch.where(ok, (d - mean) / total, 0.0), torch.where(ok, (d.abs() + size) / total, 0.0)
    ds, es = torch.zeros_like(s).scatter_add(1, at, d), torch.zeros_like(s).scatter_add(1, at, ed)
    if score == "sigmoid":
        return ds * s * (1 - s), es * s
    return s * (ds - (s * ds).sum(1, keepdim=True)), s * (es + (s * es).sum(1, keepdim=True))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 33, 32), (7, 64, 6), (3, 160, 6), (33, 256, 8), (2, 1024, 32)])
def test_backward(dg, T, E, k, dt, renorm, score):
    l, _ = _logits(T, E, dt)
    g = torch.Generator(device="cuda").manual_seed(4)
    ids, _ = _route(dg, l, k, score=score)
    ids = ids.clone()
    if T > 2:
        ids[0] = -1                                          # no choice at all
        ids[1, -1] = -1
        if k > 1:
            ids[2, 1] = ids[2, 0]                            # the same one twice
    dw = torch.randn(T, k, generator=g, device="cuda")
    buf = torch.full((T * E + 4,), 7.0, device="cuda", dtype=dt)
    dl = dg.dg_route_topk_backward(dw, l, ids, buf[:T * E].view(T, E), score=score, renormalize=renorm, factor=1.5)
    want, size = _gradient(l, ids, dw, score, renorm, 1.5)
    off = (dl.double() - want).abs()
    assert bool((off <= 2.0 ** -16 * size + R.half(dt) * want.abs() + 1e-37).all())
    assert bool((buf[T * E:] == 7).all())
    same = l.clone()
    dg.dg_route_topk_backward(dw, same, ids, same, score=score, renormalize=renorm, factor=1.5)      # in place
    assert torch.equal(same, dl)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(dg, score, renorm):
    T, E, k = 4, 40, 5
    l, _ = _logits(T, E, seed=2)
    ids, _ = _route(dg, l, k, score=score)
    g = torch.Generator(device="cuda").manual_seed(6)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dl = dg.dg_route_topk_backward(dw, l, ids, torch.empty_like(l), score=score, renormalize=renorm, factor=2.0)

    def loss(x):
        s = R.scores(x, score)
        w = torch.gather(s, 1, ids.long())
        if renorm:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return (2.0 * w * dw.double()).sum()

    for seed in range(3):
        v = torch.randn(T, E, generator=g, device="cuda", dtype=torch.float64)
        h = 2.0 ** -12
        slope = float((loss(l.double() + h * v) - loss(l.double() - h * v)) / (2 * h))
        # third derivatives of order one along v: h^2 |v|^3 < 2^-24 · 2^11
        assert abs(slope - float((dl.double() * v).sum())) <= 2.0 ** -12


def test_backward_of_saturated_sigmoids(dg):
    """s(1 - s) where s rounds to one in FP32: relative to the value itself, exp and a division for each factor below 2^-20."""
    l = torch.linspace(10.0, 40.0, 128, device="cuda").view(2, 64)
    ids = torch.arange(32, dtype=torch.int32, device="cuda").repeat(2, 1)
    dl = dg.dg_route_topk_backward(torch.ones(2, 32, device="cuda"), l, ids, torch.empty_like(l), score="sigmoid", renormalize=False)
    x = l[:, :32].double()
    want = torch.sigmoid(x) * torch.sigmoid(-x)
    assert bool(((dl[:, :32].double() - want).abs() <= 2.0 ** -20 * want).all()) and bool((dl[:, 32:] == 0).all())


def test_masked_logits_have_no_gradient(dg):
    l, _ = _logits(3, 64)
    l[:, 30:] = -torch.inf
    l[1] = -torch.inf
    for score in ("softmax", "sigmoid"):
        ids, _ = _route(dg, l, 8, score=score)
        dl = dg.dg_route_topk_backward(torch.ones(3, 8, device="cuda"), l, ids, torch.empty_like(l), score=score, renormalize=False)
        assert bool((dl[:, 30:] == 0).all()) and bool((dl[1] == 0).all()) and bool(torch.isfinite(dl).all())


def test_launch_settings_streams_and_graphs(dg, monkeypatch):
    l, b = _logits(301, 256)
    how = dict(score="sigmoid", renormalize=True, factor=2.5)
    ids, w = _route(dg, l, 8, b, **how)
    dw = torch.randn(301, 8, device="cuda")
    dl = dg.dg_route_topk_backward(dw, l, ids, torch.empty_like(l), **how)

    def same(i, x, d):
        torch.cuda.synchronize()
        return torch.equal(i, ids) and torch.equal(x, w) and torch.equal(d, dl)

    def again(stream=None):
        i, x, d = torch.empty_like(ids), torch.empty_like(w), torch.empty_like(l)
        dg.dg_route_topk(l, i, x, bias=b, stream=stream, **how)
        dg.dg_route_topk_backward(dw, l, i, d, stream=stream, **how)
        return i, x, d

    before = dg.dg_get_pdl()
    try:
        for pdl, sms in ((True, 0), (False, 0), (None, 2)):
            dg.dg_set_pdl(pdl)
            dg.dg_set_num_sms(sms)
            assert same(*again())
    finally:
        dg.dg_set_num_sms(0)
        dg.dg_set_pdl(before)
    torch.cuda.synchronize()
    assert same(*again(torch.cuda.Stream()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = again()
    for o in out:
        o.zero_()
    g.replay()
    assert same(*out)
    assert dg._bind().route(0, l, b, out[0], out[1], 1, True, 2.5, None) == 0
    monkeypatch.setattr(dg, "_bind", lambda: dg._NoBind)
    assert same(*again())
