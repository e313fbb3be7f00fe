"""The operators around the experts' products, as cases to be timed and compared.

* ``norm_fwd``: the norms at a block's boundary with its gate and residual scale, in one pass:
  R = X + gate · scale · P, P = B or B · ra · w_after (the norm after the block), and Y = R · r · W (the norm before
  the next one), as values of the stream's type and/or as E4M3 rows with 1x128 scales, the products' A operand;
* ``norm_bwd``: its backward pass: the gradients of the stream, the block's output, gate, scale and both weights;
* ``route``: the router's selection of k experts from softmax or sigmoid scores, and its backward pass;
* ``moe``: the experts' feed-forward layer for a few tokens: gate and up projections of the chosen experts,
  SwiGLU, E4M3 cast, down projection and the weighted sum over each token's experts, on E4M3 weights with
  128x128 scales (FP32 or packed UE8M0) or on four-bit weights (E2M1 with one E8M0 scale per 32);
* ``mxfp4``: the product of a few tokens with four-bit weights.

Where ``own`` is false, ``run`` computes them in elementary torch operations in FP32.
"""
import math

import torch

own = False

LIMIT = 448.0                # the largest E4M3 value
TINY = 2.0 ** -100           # the smallest group maximum that sets a scale
EPS = 1e-6


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token while decoding: the block's output joins the stream, the next products' operand comes out in FP8
        dict(name="norm token", op="norm_fwd", dtype="bf16", M=1, N=7168, block=True, after=False, gate=False, scale=False, y=False, q=True),
        # a training batch with norms on both sides of the block, gate and residual scale, statistics saved
        dict(name="norm batch", op="norm_fwd", dtype="bf16", M=8192, N=7168, block=True, after=True, gate=True, scale=True, y=True, q=False),
        # an FP32 stream of odd length, the plain norm before a block in both forms
        dict(name="norm odd", op="norm_fwd", dtype="f32", M=4099, N=2112, block=False, after=False, gate=False, scale=False, y=True, q=True),
        # a small layer's backward pass, where launches count
        dict(name="norm bwd small", op="norm_bwd", dtype="bf16", M=200, N=1024, block=True, after=False, gate=False, scale=True),
        # the full batch's backward pass, every gradient
        dict(name="norm bwd batch", op="norm_bwd", dtype="bf16", M=8192, N=7168, block=True, after=True, gate=True, scale=True),
        # a prefill or training batch's routing: sigmoid scores, a balancing bias in the selection alone
        dict(name="route batch", op="route", pass_="fwd", T=16384, E=256, k=8, score="sigmoid", bias=True, renorm=True, factor=2.5),
        # its backward pass for softmax scores that are not normalised again: every logit gets a gradient
        dict(name="route bwd", op="route", pass_="bwd", T=16381, E=160, k=6, score="softmax", bias=False, renorm=False, factor=1.0),
        # one token through the routed experts
        dict(name="moe token", op="moe", weights="fp32", T=1, k=8, E=32, K=7168, I=2048),
        # a small decoding batch: most experts have a token or two
        dict(name="moe batch", op="moe", weights="ue8m0", T=16, k=8, E=64, K=7168, I=2048),
        # a narrower layer with four-bit experts, odd sizes, a token without experts
        dict(name="moe four-bit", op="moe", weights="mxfp4", T=5, k=4, E=16, K=2080, I=1408),
        # one token through a large projection kept in four bits
        dict(name="mxfp4 token", op="mxfp4", M=1, N=7168, K=16384),
        # a small batch through a projection
        dict(name="mxfp4 batch", op="mxfp4", M=16, N=24576, K=1536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "route", "moe", "moe", "mxfp4"])
    if op in ("norm_fwd", "norm_bwd"):
        block = rng.random() < 0.75
        case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), M=_log(rng, 1, 4096), N=16 * _log(rng, 2, 448) - rng.choice([0, 0, 3]),
                    block=block, after=block and rng.random() < 0.5, gate=block and rng.random() < 0.5, scale=block and rng.random() < 0.5)
        if op == "norm_fwd":
            case["q"] = case["N"] % 16 == 0 and rng.random() < 0.6
            case["y"] = not case["q"] or rng.random() < 0.5
        return case
    if op == "route":
        E = _log(rng, 8, 512)
        return dict(op=op, pass_=rng.choice(["fwd", "bwd"]), T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 10)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, renorm=rng.random() < 0.5,
                    factor=rng.choice([1.0, 1.0, 2.5]))
    if op == "mxfp4":
        return dict(op=op, M=_log(rng, 1, 24), N=8 * _log(rng, 8, 1024), K=32 * _log(rng, 4, 256))
    E = _log(rng, 4, 64)
    return dict(op=op, weights=rng.choice(["fp32", "ue8m0", "mxfp4"]), T=_log(rng, 1, 16), k=rng.randint(1, min(E, 8)), E=E,
                K=32 * _log(rng, 8, 160), I=128 * rng.randint(1, 12))


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, size = case["M"] * case["N"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm_fwd":
            return {"bytes": n * (size * (1 + 2 * case["block"] + case["y"]) + case["q"]), "flops": n * (8 if case["block"] else 4)}
        return {"bytes": n * size * (4 + 2 * case["block"]), "flops": n * (24 if case["block"] else 10)}
    if op == "route":
        n = case["T"] * case["E"]
        return {"bytes": 4 * n * (2 if case["pass_"] == "bwd" else 1) + 8 * case["T"] * case["k"], "flops": 8 * n}
    bits = lambda fmt: 4.25 if fmt == "mxfp4" else 8.0     # noqa: E731
    if op == "mxfp4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": int(N * K * bits("mxfp4") / 8) + M * K + 2 * M * N, "flops": 2 * M * N * K}
    T, k, E, K, I = (case[n] for n in ("T", "k", "E", "K", "I"))
    active = E * (1.0 - (1.0 - k / E) ** T)                # of experts chosen evenly
    return {"bytes": int(active * 3 * I * K * bits(case["weights"]) / 8) + 3 * T * K, "flops": 6 * T * k * I * K}


# -------------------------------------------------------------------------------------- FP8 and FP4

def _pow2(amax):
    """The smallest power of two s with amax / s <= 448."""
    m, e = torch.frexp(amax)                       # amax = m · 2^e, m in [1/2, 1); 448 = 7/8 · 2^9
    return torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))


def _groups(y, gr, gc):
    """[.., M, N] -> [.., Mb, gr, Nb, gc], zeros past the end."""
    M, N = y.shape[-2:]
    Mb, Nb = _cdiv(M, gr), _cdiv(N, gc)
    out = y.new_zeros(y.shape[:-2] + (Mb * gr, Nb * gc))
    out[..., :M, :N] = y
    return out.unflatten(-1, (Nb, gc)).unflatten(-3, (Mb, gr))


def _cast(y, gr, gc, pow2):
    """y [.., M, N] -> E4M3 codes and the scales [.., ceil(M/gr), ceil(N/gc)] of its gr x gc groups."""
    M, N = y.shape[-2:]
    g = _groups(y, gr, gc)
    amax = g.abs().amax(dim=(-3, -1))
    a = amax.clamp_min(TINY)
    s = _pow2(a) if pow2 else a / LIMIT
    f = 1.0 / s if pow2 else LIMIT / a
    one = torch.ones_like(a)
    s, f = torch.where(amax > 0, s, one), torch.where(amax > 0, f, one)
    q = (g * f[..., :, None, :, None]).clamp(-LIMIT, LIMIT).flatten(-4, -3).flatten(-2, -1)[..., :M, :N]
    return q.contiguous().to(torch.float8_e4m3fn), s


def _spread(s, gr, gc, M, N):
    """The scales of gr x gc groups at every element of [.., M, N]."""
    return s.repeat_interleave(gr, -2)[..., :M, :].repeat_interleave(gc, -1)[..., :N]


def _pack(s):
    """Power-of-two scales [.., n] -> their E8M0 codes, four to an int32 word; 127 past the end."""
    n = s.shape[-1]
    codes = s.new_full(s.shape[:-1] + (4 * _cdiv(n, 4),), 127.0)
    codes[..., :n] = torch.frexp(s)[1].to(s.dtype) + 126
    return codes.to(torch.uint8).contiguous().view(torch.int32)


def _unpack(w, n):
    codes = w.contiguous().view(torch.uint8)[..., :n]
    return torch.ldexp(torch.ones(codes.shape, device=w.device), codes.to(torch.int32) - 127)


def _lay_rows(s, pow2):
    """Scales [M, n] of 1x128 groups in the products' layout: [n, align4(M)] with zeros, or packed words."""
    M, ld = s.shape[0], 4 * _cdiv(s.shape[0], 4)
    full = s.new_full((ld, s.shape[1]), 1.0 if pow2 else 0.0)
    full[:M] = s
    return _pack(full).t().contiguous() if pow2 else full.t().contiguous()


def _four_bits(w):
    """w [.., K] -> E2M1 codes two to a byte (the even k in the low half) and E8M0 scales of groups of 32."""
    g = w.unflatten(-1, (-1, 32))
    e = torch.frexp(g.abs().amax(-1).clamp_min(2.0 ** -100))[1] - 3       # the largest magnitude falls into [4, 8)
    v = g / torch.ldexp(torch.ones_like(e, dtype=w.dtype), e)[..., None]
    ends = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = (torch.bucketize(v.abs(), ends) + 8 * (v < 0)).to(torch.uint8).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _four_bit_values(q, s):
    """The values of E2M1 codes [.., K/2] with E8M0 scales [.., K/32]."""
    code = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2).long()
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    v = table[code & 7] * (1.0 - 2.0 * (code >> 3))
    return v * torch.ldexp(torch.ones(s.shape, device=q.device), s.to(torch.int32) - 127).repeat_interleave(32, -1)


# ------------------------------------------------------------------------------------------- inputs

def _activations(gen, M, N):
    """Like a normalised residual stream: unit variance, a few channels several times larger."""
    x = torch.randn(M, N, generator=gen, device="cuda")
    loud = torch.rand(N, generator=gen, device="cuda") < 0.01
    return x * torch.where(loud, 6.0, 1.0)


def _choices(gen, T, E, k):
    """Experts of each token from uneven popularities, and their weights; of several tokens the last has none."""
    logits = torch.randn(T, E, generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    w = torch.softmax(top[:, :k], dim=1)
    ids = ids[:, :k].to(torch.int32)
    if T > 4:
        ids[-1], w[-1] = -1, 0.0
    return ids.contiguous(), w.contiguous()


def _expert_weights(gen, E, N, K, fmt):
    """[E, N, K] weights in their stored form, some experts at a time."""
    parts = []
    for at in range(0, E, 8):
        w = torch.randn(min(8, E - at), N, K, generator=gen, device="cuda") * (1.0 / math.sqrt(K))
        if fmt == "mxfp4":
            parts.append(_four_bits(w))
        else:
            q, s = _cast(w, 128, 128, fmt == "ue8m0")
            parts.append((q, _pack(s) if fmt == "ue8m0" else s))
    return tuple(torch.cat(p) for p in zip(*[(q.view(torch.uint8), s) for q, s in parts]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")      # noqa: E731
    op, st = case["op"], {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        M, N = case["M"], case["N"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        empty = lambda: torch.empty(M, N, dtype=dt, device="cuda")                # noqa: E731
        f32 = lambda *shape: torch.empty(*shape, device="cuda")                   # noqa: E731
        x = _activations(gen, M, N)
        st["W"] = 1.0 + 0.2 * randn(N)
        st["B"] = (0.3 * randn(M, N)).to(dt) if case["block"] else None
        st["w_after"] = 1.0 + 0.2 * randn(N) if case["after"] else None
        st["gate"] = torch.sigmoid(randn(M)) if case["gate"] else None
        st["scale"] = 0.1 + 0.02 * randn(N) if case["scale"] else None
        if op == "norm_fwd":
            st["X"] = x.to(dt)
            st["R"] = empty() if case["block"] else None
            st["Y"] = empty() if case["y"] else None
            st["Yq"] = torch.empty(M, N, dtype=torch.float8_e4m3fn, device="cuda") if case["q"] else None
            st["sY"] = f32(_cdiv(N, 128), 4 * _cdiv(M, 4)) if case["q"] else None
            st["rstd"], st["rstd_after"] = f32(M), f32(M) if case["after"] else None
        else:
            st["R"] = x.to(dt)
            st["dY"], st["dR"] = (0.02 * randn(M, N)).to(dt), (0.02 * randn(M, N)).to(dt)
            st["rstd"] = (st["R"].double().square().mean(1) + EPS).rsqrt().float()
            st["rstd_after"] = (st["B"].double().square().mean(1) + EPS).rsqrt().float() if case["after"] else None
            st["dX"], st["dW"] = empty(), f32(N)
            st["dB"] = empty() if case["block"] else None
            st["dw_after"] = f32(N) if case["after"] else None
            st["dgate"] = f32(M) if case["gate"] else None
            st["dscale"] = f32(N) if case["scale"] else None
        return st
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = 1.5 * randn(T, E) + 0.5 * randn(E)
        st["bias"] = 0.1 * randn(E) if case["bias"] else None
        st["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty(T, k, device="cuda")
        if case["pass_"] == "bwd":
            st["ids"] = torch.argsort(st["logits"], dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
            st["dweights"], st["dlogits"] = 0.1 * randn(T, k), torch.empty(T, E, device="cuda")
        return st
    M, K = case["M" if op == "mxfp4" else "T"], case["K"]
    pow2 = case.get("weights") == "ue8m0"
    st["A"], sa = _cast(_activations(gen, M, K).to(torch.bfloat16).float(), 1, 128, pow2)
    st["sA"] = _lay_rows(sa, pow2)
    if op == "mxfp4":
        st["B"], st["sB"] = _four_bits(randn(case["N"], K) * (1.0 / math.sqrt(K)))
        st["D"] = torch.empty(M, case["N"], dtype=torch.bfloat16, device="cuda")
        return st
    E, I, fmt = case["E"], case["I"], case["weights"]
    st["W1"], st["sW1"] = _expert_weights(gen, E, 2 * I, K, fmt)
    st["W2"], st["sW2"] = _expert_weights(gen, E, K, I, fmt)
    st["ids"], st["weights"] = _choices(gen, M, E, case["k"])
    st["Y"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    return st


# ---------------------------------------------------------------------------------------- the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm_fwd": _own_norm, "norm_bwd": _own_norm_bwd, "route": _own_route, "moe": _own_moe, "mxfp4": _own_mxfp4}[op](state)
    return {"norm_fwd": _plain_norm, "norm_bwd": _plain_norm_bwd, "route": _plain_route, "moe": _plain_moe, "mxfp4": _plain_mxfp4}[op](state)


def _own_norm(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    names = ("R", "Y", "Yq", "sY", "rstd", "rstd_after")
    dg.dg_residual_norm(st["X"], st["W"], B=st["B"], w_after=st["w_after"], gate=st["gate"], scale=st["scale"], eps=EPS,
                        **{n: st[n] for n in names})
    return {n: st[n] for n in names}


def _own_norm_bwd(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    names = ("dX", "dW", "dB", "dw_after", "dgate", "dscale")
    dg.dg_residual_norm_backward(st["dY"], st["R"], st["rstd"], st["W"], dR=st["dR"], B=st["B"], rstd_after=st["rstd_after"],
                                 w_after=st["w_after"], gate=st["gate"], scale=st["scale"], **{n: st[n] for n in names})
    return {n: st[n] for n in names}


def _own_route(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    case = st["case"]
    how = dict(score=case["score"], renormalize=case["renorm"], factor=case["factor"])
    if case["pass_"] == "bwd":
        return dg.dg_route_topk_backward(st["dweights"], st["logits"], st["ids"], st["dlogits"], **how)
    dg.dg_route_topk(st["logits"], st["ids"], st["weights"], bias=st["bias"], **how)
    return {"ids": st["ids"], "weights": st["weights"]}


def _own_moe(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    call = {"fp32": dg.dg_fp8_moe_swiglu, "ue8m0": dg.dg_fp8_moe_swiglu_ue8m0, "mxfp4": dg.dg_fp8_moe_swiglu_mxfp4}[st["case"]["weights"]]
    return call(st["A"], st["sA"], st["W1"], st["sW1"], st["W2"], st["sW2"], st["ids"], st["weights"], st["Y"])


def _own_mxfp4(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    return dg.dg_fp8_mxfp4_gemm_nt(st["A"], st["sA"], st["B"], st["sB"], st["D"])


def _plain_norm(st):
    case, dt, r = st["case"], st["X"].dtype, st["X"].float()
    out = {"R": None, "Y": None, "Yq": None, "sY": None, "rstd_after": None}
    if case["block"]:
        p = st["B"].float()
        if case["after"]:
            out["rstd_after"] = 1.0 / torch.sqrt(p.square().mean(1) + EPS)
            p = p * out["rstd_after"][:, None] * st["w_after"]
        if case["gate"]:
            p = p * st["gate"][:, None]
        if case["scale"]:
            p = p * st["scale"]
        r = r + p
        out["R"] = r.to(dt)
    out["rstd"] = 1.0 / torch.sqrt(r.square().mean(1) + EPS)
    y = r * out["rstd"][:, None] * st["W"]
    if case["y"]:
        out["Y"] = y.to(dt)
    if case["q"]:
        out["Yq"], s = _cast(y, 1, 128, False)
        out["sY"] = _lay_rows(s, False)
    return out


def _plain_norm_bwd(st):
    case, dt = st["case"], st["R"].dtype
    dy, xh = st["dY"].float(), st["R"].float() * st["rstd"][:, None]
    gw = dy * st["W"]
    g = st["dR"].float() + st["rstd"][:, None] * (gw - xh * (gw * xh).mean(1, keepdim=True))
    out = {"dX": g.to(dt), "dW": (dy * xh).sum(0), "dB": None, "dw_after": None, "dgate": None, "dscale": None}
    if not case["block"]:
        return out
    b = st["B"].float()
    bh = b * st["rstd_after"][:, None] if case["after"] else b
    p = bh * st["w_after"] if case["after"] else b
    gate = st["gate"][:, None] if case["gate"] else torch.ones(1, 1, device=b.device)
    scale = st["scale"] if case["scale"] else torch.ones(1, device=b.device)
    if case["gate"]:
        out["dgate"] = (scale * p * g).sum(1)
    if case["scale"]:
        out["dscale"] = (gate * p * g).sum(0)
    q = gate * scale * g
    if case["after"]:
        out["dw_after"] = (q * bh).sum(0)
        qw = q * st["w_after"]
        q = st["rstd_after"][:, None] * (qw - bh * (qw * bh).mean(1, keepdim=True))
    out["dB"] = q.to(dt)
    return out


def _scores(logits, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(st):
    case, l = st["case"], st["logits"]
    s = _scores(l, case["score"])
    if case["pass_"] == "fwd":
        # the selection in 64 bits: scores next to the border of the k-th
        key = l if st["bias"] is None else _scores(l.double(), case["score"]) + st["bias"].double()
        ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :case["k"]]
        w = torch.gather(s, 1, ids)
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return {"ids": ids.to(torch.int32), "weights": w * case["factor"]}
    ids, dw = st["ids"].long(), st["dweights"] * case["factor"]
    if case["renorm"]:
        sel = torch.gather(s, 1, ids)
        total = sel.sum(1, keepdim=True) + 1e-20
        dw = (dw - (dw * sel).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_add(1, ids, dw)
    return ds * s * (1.0 - s) if case["score"] == "sigmoid" else s * (ds - (s * ds).sum(1, keepdim=True))


def _row_values(q, s, pow2):
    """The values of E4M3 rows with scales in the products' layout."""
    M, K = q.shape
    s = _unpack(s.t(), _cdiv(K, 128))[:M] if pow2 else s.t()[:M]
    return q.float() * _spread(s, 1, 128, M, K)


def _weight_values(q, s, fmt):
    """The values of stored weights [.., N, K]."""
    if fmt == "mxfp4":
        return _four_bit_values(q, s)
    N, K = q.shape[-2:]
    s = _unpack(s, _cdiv(K, 128)) if fmt == "ue8m0" else s
    return q.view(torch.float8_e4m3fn).float() * _spread(s, 128, 128, N, K)


def _plain_moe(st):
    case, fmt, ids, w = st["case"], st["case"]["weights"], st["ids"], st["weights"]
    T, k, E, I = case["T"], case["k"], case["E"], case["I"]
    x = _row_values(st["A"], st["sA"], fmt == "ue8m0")
    if T * k <= E:      # the experts of each (token, choice), else all of them
        at = ids.flatten().clamp_min(0).long()
        mix = torch.zeros(T * k, T, device=x.device)
        mix[torch.arange(T * k, device=x.device), torch.arange(T * k, device=x.device) // k] = torch.where(ids >= 0, w, torch.zeros_like(w)).flatten()
    else:
        at = torch.arange(E, device=x.device)
        mix = ((ids[None] == at[:, None, None]) * w).sum(2)                     # [E, T]
    d = torch.matmul(x, _weight_values(st["W1"][at], st["sW1"][at], fmt).transpose(1, 2))    # [S, T, 2I]
    g, u = d[..., :I], d[..., I:]
    h = g / (1.0 + torch.exp(-g)) * u
    q, s = _cast(h, 1, 128, fmt == "ue8m0")
    h = q.float() * _spread(s, 1, 128, T, I)
    y = torch.matmul(h, _weight_values(st["W2"][at], st["sW2"][at], fmt).transpose(1, 2))    # [S, T, K]
    return (y * mix[..., None]).sum(0).to(torch.bfloat16)


def _plain_mxfp4(st):
    return (_row_values(st["A"], st["sA"], False) @ _four_bit_values(st["B"], st["sB"]).t()).to(torch.bfloat16)


# ------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_fwd": _exact_norm, "norm_bwd": _exact_norm_bwd, "route": _exact_route, "moe": _exact_moe, "mxfp4": _exact_mxfp4}[case["op"]](st)


def _of(st, name, like):
    """A vector of the state in 64 bits, or ones."""
    return torch.ones(like, dtype=torch.float64, device="cuda") if st[name] is None else st[name].double()


def _exact_codes(v):
    """The codes' values (before their rounding to E4M3) and scales of 1x128 groups of v [M, N]."""
    M, N = v.shape
    codes, scales = torch.empty_like(v), torch.zeros(_cdiv(N, 128), 4 * _cdiv(M, 4), dtype=torch.float64, device=v.device)
    for b, part in enumerate(v.split(128, 1)):
        top = part.abs().amax(1)
        s = torch.where(top > 0, top.clamp_min(TINY) / LIMIT, torch.ones_like(top))
        codes[:, b * 128:b * 128 + part.shape[1]] = part / s[:, None]
        scales[b, :M] = s
    return codes, scales


def _exact_norm(st):
    case = st["case"]
    M, N = case["M"], case["N"]
    r, ra = st["X"].double(), None
    if case["block"]:
        b = st["B"].double()
        if case["after"]:
            ra = (torch.einsum("mn,mn->m", b, b) / N + EPS) ** -0.5
            b = torch.einsum("mn,m,n->mn", b, ra, _of(st, "w_after", N))
        r = r + torch.einsum("mn,m,n->mn", b, _of(st, "gate", M), _of(st, "scale", N))
    rstd = (torch.einsum("mn,mn->m", r, r) / N + EPS) ** -0.5
    y = torch.einsum("mn,m,n->mn", r, rstd, st["W"].double())
    codes, scales = _exact_codes(y) if case["q"] else (None, None)
    return {"R": r if case["block"] else None, "Y": y if case["y"] else None, "Yq": codes, "sY": scales, "rstd": rstd, "rstd_after": ra}


def _exact_norm_of(u, x, rs, w):
    """The gradient of x · rs(x) · w for the outer gradient u: (of x, of w). rs: the reciprocal root of x's mean square."""
    t = torch.einsum("mn,n->mn", u, w)
    along = torch.einsum("mn,mn,m->m", t, x, rs ** 3) / x.shape[1]
    return t * rs[:, None] - x * along[:, None], torch.einsum("mn,mn,m->n", u, x, rs)


def _exact_norm_bwd(st):
    case = st["case"]
    M, N = case["M"], case["N"]
    dx, dw = _exact_norm_of(st["dY"].double(), st["R"].double(), st["rstd"].double(), st["W"].double())
    dx = dx + st["dR"].double()
    out = {"dX": dx, "dW": dw, "dB": None, "dw_after": None, "dgate": None, "dscale": None}
    if not case["block"]:
        return out
    gate, scale, b = _of(st, "gate", M), _of(st, "scale", N), st["B"].double()
    p = torch.einsum("mn,m,n->mn", b, _of(st, "rstd_after", M), _of(st, "w_after", N))
    if case["gate"]:
        out["dgate"] = torch.einsum("mn,mn,n->m", dx, p, scale)
    if case["scale"]:
        out["dscale"] = torch.einsum("mn,mn,m->n", dx, p, gate)
    dp = torch.einsum("mn,m,n->mn", dx, gate, scale)
    if case["after"]:
        out["dB"], out["dw_after"] = _exact_norm_of(dp, b, st["rstd_after"].double(), st["w_after"].double())
    else:
        out["dB"] = dp
    return out


def _exact_route(st):
    case, l = st["case"], st["logits"].double()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    if case["pass_"] == "fwd":
        left = (l if st["bias"] is None else s + st["bias"].double()).clone()
        ids, ws = [], []
        for _ in range(case["k"]):
            top = left.amax(1, keepdim=True)
            at = torch.where(left == top, torch.arange(case["E"], device=l.device), case["E"]).amin(1, keepdim=True)
            ids.append(at)
            ws.append(torch.gather(s, 1, at))
            left.scatter_(1, at, -math.inf)
        w = torch.cat(ws, 1)
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return {"ids": torch.cat(ids, 1).to(torch.int32), "weights": case["factor"] * w}
    l.requires_grad_()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    w = torch.gather(s, 1, st["ids"].long())
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return torch.autograd.grad(w, l, case["factor"] * st["dweights"].double())[0]


def _exact_e8m0(w, n):
    """Packed E8M0 scales in 64 bits, byte by byte."""
    b = torch.stack([(w >> (8 * j)) & 0xFF for j in range(4)], dim=-1).flatten(-2)[..., :n]
    return torch.pow(2.0, b.double() - 127.0)


def _exact_rows(st, pow2):
    M, K = st["A"].shape
    s = _exact_e8m0(st["sA"].t(), _cdiv(K, 128)) if pow2 else st["sA"].t().double()
    return st["A"].double() * s[:M][:, torch.arange(K, device=s.device) // 128]


def _exact_weights(q, s, fmt):
    """One matrix of stored weights [N, K] in 64 bits, at every element's own place."""
    if fmt == "mxfp4":
        N, K = q.shape[0], 2 * q.shape[1]
        at = torch.arange(K, device=q.device)
        code = (q.long()[:, at // 2] >> (4 * (at % 2))) & 15
        e, m = (code >> 1) & 3, (code & 1).double()
        v = torch.where(e > 0, (1.0 + m / 2) * torch.pow(2.0, (e - 1).double()), m / 2)
        return torch.where(code >= 8, -v, v) * torch.pow(2.0, s.double() - 127.0)[:, at // 32]
    N, K = q.shape
    s = _exact_e8m0(s, _cdiv(K, 128)) if fmt == "ue8m0" else s.double()
    rows, cols = torch.arange(N, device=q.device) // 128, torch.arange(K, device=q.device) // 128
    return q.view(torch.float8_e4m3fn).double() * s[rows][:, cols]


def _exact_moe(st):
    case, fmt = st["case"], st["case"]["weights"]
    I, pow2 = case["I"], case["weights"] == "ue8m0"
    x = _exact_rows(st, pow2)
    y = torch.zeros_like(x)
    ids, w = st["ids"].tolist(), st["weights"].double()
    for e in sorted({i for row in ids for i in row if i >= 0}):
        places = [(t, j) for t, row in enumerate(ids) for j, i in enumerate(row) if i == e]
        ts, js = [t for t, _ in places], [j for _, j in places]
        d = x[ts] @ _exact_weights(st["W1"][e], st["sW1"][e], fmt).t()
        h = d[:, :I] * torch.sigmoid(d[:, :I]) * d[:, I:]
        for part in h.split(128, 1):             # the cast that the operator's definition makes
            top = part.abs().amax(1, keepdim=True)
            s = torch.where(top > 0, top.clamp_min(TINY) / LIMIT, torch.ones_like(top))
            if pow2:
                s = torch.pow(2.0, torch.ceil(torch.log2(s)))     # (h is never at a border to 64 bits)
            part.copy_((part / s).clamp(-LIMIT, LIMIT).float().to(torch.float8_e4m3fn).double() * s)
        y.index_add_(0, torch.tensor(ts, device=x.device), (h @ _exact_weights(st["W2"][e], st["sW2"][e], fmt).t()) * w[ts, js][:, None])
    return y


def _exact_mxfp4(st):
    return _exact_rows(st, False) @ _exact_weights(st["B"], st["sB"], "mxfp4").t()
