"""The training operators of the expert feed-forward layer, as cases to be timed and compared.

Four operators, each in the form a training or serving program calls it:

* ``ffn_fwd``: the gated projection H = dropout(silu(X Wgᵀ) · (X Wuᵀ)) on FP8 operands with fine-grained
  scales, dense or over contiguous expert groups, the pre-activations [X Wgᵀ | X Wuᵀ] saved on request;
* ``ffn_bwd``: its backward pass. The gradients of the pre-activations are cast to E4M3 along both
  contractions (1x128 groups of each token's features, 128x1 groups of tokens), as the definition of the
  operator says, and give dX = dGU·W and dW = dGUᵀ·X;
* ``dropout``: dropout from a counter-based generator (Philox4x32-10, 16 bits an element) and the
  residual sum, its mask never stored; the backward pass is the same call on the gradient;
* ``cast``: BF16 to E4M3 with one scale per 1x128, 128x1 or 128x128 group, the forms the products read.

Where ``own`` is false, ``run`` computes them in elementary torch operations in FP32.
"""
import math
import random

import torch

own = False

LIMIT = 448.0                # the largest E4M3 value
TINY = 2.0 ** -100           # the smallest group maximum that sets a scale


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through the up/gate projection while serving: the weights' read and the launch count
        dict(name="fwd token", op="ffn_fwd", layout="dense", scales="fp32", M=1, I=2048, K=7168, G=1, p=0.0, save=False),
        # a short, odd batch of a narrow layer whose K is no multiple of 128
        dict(name="fwd odd", op="ffn_fwd", layout="dense", scales="ue8m0", M=333, I=1152, K=2064, G=1, p=0.0, save=True),
        # a full training (or prefill) batch of a dense or shared expert
        dict(name="fwd batch", op="ffn_fwd", layout="dense", scales="fp32", M=4096, I=2048, K=7168, G=1, p=0.0, save=True),
        # routed experts while fine-tuning: ragged groups, one of them empty, dropout inside the experts
        dict(name="fwd experts", op="ffn_fwd", layout="grouped", scales="ue8m0", M=8192, I=2048, K=7168, G=8, p=0.1, save=True),
        # a small layer's backward pass, where launches count
        dict(name="bwd small", op="ffn_bwd", layout="dense", scales="fp32", M=200, I=512, K=1024, G=1, p=0.0, save=True),
        # the full batch's backward pass
        dict(name="bwd batch", op="ffn_bwd", layout="dense", scales="fp32", M=4096, I=2048, K=7168, G=1, p=0.0, save=True),
        # the routed experts' backward pass, with the dropout of the forward pass made again
        dict(name="bwd experts", op="ffn_bwd", layout="grouped", scales="ue8m0", M=8192, I=2048, K=7168, G=8, p=0.1, save=True),
        # the residual sum of a few tokens
        dict(name="dropout few", op="dropout", dtype="bf16", rows=64, cols=2112, p=0.1, residual=True),
        # the residual sum of a full batch
        dict(name="dropout batch", op="dropout", dtype="bf16", rows=16384, cols=7168, p=0.1, residual=True),
        # a gradient in FP32 of odd length
        dict(name="dropout odd", op="dropout", dtype="f32", rows=4099, cols=2113, p=0.5, residual=False),
        # the activations of a serving batch, for the forward product alone
        dict(name="cast few", op="cast", scales="fp32", M=64, N=7168, rows=True, cols=False, blocks=False),
        # the activations of a training batch: rows for the products, 128x1 groups and blocks for the weight gradients
        dict(name="cast batch", op="cast", scales="ue8m0", M=8192, N=7168, rows=True, cols=True, blocks=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_fwd", "ffn_bwd", "ffn_bwd", "dropout", "cast"])
    scales = rng.choice(["fp32", "ue8m0"])
    if op == "dropout":
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), rows=_log(rng, 1, 8192), cols=_log(rng, 16, 7168),
                    p=rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]), residual=rng.random() < 0.5)
    if op == "cast":
        form = rng.choice([(True, False, False), (True, True, False), (True, True, True), (False, False, True), (True, False, True)])
        return dict(op=op, scales=scales, M=_log(rng, 1, 8192), N=16 * _log(rng, 2, 448), rows=form[0], cols=form[1], blocks=form[2])
    layout = rng.choice(["dense", "grouped"])
    return dict(op=op, layout=layout, scales=scales, M=_log(rng, 1 if layout == "dense" else 16, 4096),
                I=128 * _log(rng, 1, 16), K=16 * _log(rng, 8, 448), G=1 if layout == "dense" else rng.randint(2, 16),
                p=rng.choice([0.0, 0.0, 0.1, 0.3]), save=op == "ffn_bwd" or rng.random() < 0.7)


def _cdiv(a, b):
    return -(-a // b)


def _rows(case):
    """Rows of the token buffers. Grouped: a static buffer, which holds any split of the tokens into
    groups that are each padded to 128 rows."""
    return case["M"] if case["layout"] == "dense" else 128 * (_cdiv(case["M"], 128) + case["G"])


def work(case):
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2 * n}
    if case["op"] == "cast":
        n = case["M"] * case["N"]
        forms = case["rows"] + case["cols"] + case["blocks"]
        return {"bytes": 2 * n + forms * n, "flops": 2 * n * forms}
    M, I, K, G = case["M"], case["I"], case["K"], case["G"]
    if case["op"] == "ffn_fwd":
        return {"bytes": M * K + G * 2 * I * K + 2 * M * I * (3 if case["save"] else 1), "flops": 4 * M * I * K}
    return {"bytes": 2 * M * I * 3 + G * 2 * I * K + M * K + 2 * M * K + 2 * G * 2 * I * K, "flops": 8 * M * I * K}


# ------------------------------------------------------------------------------------- the FP8 cast

def _pow2(amax):
    """The smallest power of two s with amax / s <= 448."""
    m, e = torch.frexp(amax)                       # amax = m · 2^e, m in [1/2, 1); 448 = 7/8 · 2^9
    return torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))


def _factors(amax, scales):
    """(factor to codes, scale back) of groups with these maxima."""
    a = amax.clamp_min(TINY)
    s = _pow2(a) if scales == "ue8m0" else a / LIMIT
    f = 1.0 / s if scales == "ue8m0" else LIMIT / a
    one = torch.ones_like(a)
    return torch.where(amax > 0, f, one), torch.where(amax > 0, s, one)


def _pad(x, rows, cols):
    out = x.new_zeros(x.shape[:-2] + (rows, cols))
    out[..., :x.shape[-2], :x.shape[-1]] = x
    return out


def _cast(x, gr, gc, scales):
    """x [.., M, N] -> E4M3 codes [.., M, N] and the scales [.., ceil(M/gr), ceil(N/gc)] of its gr x gc groups."""
    M, N = x.shape[-2:]
    Mb, Nb = _cdiv(M, gr), _cdiv(N, gc)
    y = _pad(x, Mb * gr, Nb * gc).unflatten(-1, (Nb, gc)).unflatten(-3, (Mb, gr))     # [.., Mb, gr, Nb, gc]
    f, s = _factors(y.abs().amax(dim=(-3, -1)), scales)
    q = (y * f[..., :, None, :, None]).clamp(-LIMIT, LIMIT).flatten(-4, -3).flatten(-2, -1)[..., :M, :N]
    return q.contiguous().to(torch.float8_e4m3fn), s


def _spread(s, gr, gc, M, N):
    """The scales of gr x gc groups at every element of [.., M, N]."""
    return s.repeat_interleave(gr, -2)[..., :M, :].repeat_interleave(gc, -1)[..., :N]


def _pack(s):
    """Power-of-two scales [.., n] -> their E8M0 codes, four to an int32 word [.., ceil(n/4)]; 127 past the end."""
    n = s.shape[-1]
    codes = s.new_full(s.shape[:-1] + (4 * _cdiv(n, 4),), 127.0)
    codes[..., :n] = torch.frexp(s)[1].to(s.dtype) + 126
    return codes.to(torch.uint8).contiguous().view(torch.int32)


def _unpack(w, n):
    codes = w.contiguous().view(torch.uint8)[..., :n]
    return torch.ldexp(torch.ones(codes.shape, device=w.device), codes.to(torch.int32) - 127)


def _lay_rows(s, scales):
    """Scales [M, n] of 1x128 groups in the products' layout: [n, align4(M)], or packed words."""
    M, ld = s.shape[0], 4 * _cdiv(s.shape[0], 4)
    if scales == "ue8m0":
        full = torch.ones(ld, s.shape[1], device=s.device)
        full[:M] = s
        return _pack(full).t().contiguous()
    return _pad(s, ld, s.shape[1]).t().contiguous()


def _lay_last(s, scales):
    """Scales whose last axis runs along the contraction."""
    return _pack(s) if scales == "ue8m0" else s.contiguous()


def _unlay_rows(s, M, n, scales):
    return _unpack(s.t(), n)[:M] if scales == "ue8m0" else s.t()[:M]


def _unlay_last(s, n, scales):
    return _unpack(s, n) if scales == "ue8m0" else s


# ------------------------------------------------------------------------------------ the generator

def _philox(index, seed, offset):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC'11) of the counters (index, offset) under the key
    `seed`: four 32-bit words each, in int64."""
    low = 0xFFFFFFFF
    c0, c1 = index & low, (index >> 32) & low
    c2, c3 = torch.full_like(index, offset & low), torch.full_like(index, (offset >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], dim=-1)


def _threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def _keep(n, p, rng, device):
    """Whether each of n elements is kept: element i has the 16 bits i % 8 of counter i // 8."""
    words = _philox(torch.arange(_cdiv(n, 8), device=device), *rng)
    halves = torch.stack([words & 0xFFFF, words >> 16], dim=-1).reshape(-1)[:n]
    return halves >= _threshold(p)


def _keep_scale(p):
    t = _threshold(p)
    return 65536.0 / (65536.0 - t) if t < 65536 else 0.0


def _dropped(x, p, rng):
    if p == 0:
        return x
    keep = _keep(x.numel(), p, rng, x.device).view(x.shape)
    return torch.where(keep, x * _keep_scale(p), torch.zeros_like(x))


# ------------------------------------------------------------------------------------------- inputs

def _activations(gen, M, N, device):
    """Like a normalised residual stream: unit variance, a few channels several times larger."""
    x = torch.randn(M, N, generator=gen, device=device)
    loud = torch.rand(N, generator=gen, device=device) < 0.01
    return (x * torch.where(loud, 6.0, 1.0)).to(torch.bfloat16)


def _groups(case, seed):
    """Tokens of each expert: uneven, and now and then none."""
    rng, G = random.Random(seed * 7919 + 17), case["G"]
    weight = [rng.uniform(0.2, 1.0) for _ in range(G)]
    weight[rng.randrange(G)] = 0.0
    cuts, at, total = [], 0.0, sum(weight)
    for w in weight:
        at += w
        cuts.append(int(round(case["M"] * at / total)))
    cuts[-1] = case["M"]
    return [b - a for a, b in zip([0] + cuts, cuts)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = (random.Random(seed).getrandbits(62), seed % 1000003)
    st = {"case": case, "rng": rng, "rng_dev": torch.tensor(rng, dtype=torch.int64, device=dev)}
    if case["op"] == "dropout":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        shape = (case["rows"], case["cols"])
        st["x"] = torch.randn(shape, generator=gen, device=dev).to(dt)
        st["r"] = torch.randn(shape, generator=gen, device=dev).to(dt) if case["residual"] else None
        st["y"] = torch.empty(shape, dtype=dt, device=dev)
        return st
    scales = case["scales"]
    sdt = torch.int32 if scales == "ue8m0" else torch.float32
    words = (lambda n: _cdiv(n, 4)) if scales == "ue8m0" else (lambda n: n)
    if case["op"] == "cast":
        M, N = case["M"], case["N"]
        Mb, Nb, ld = _cdiv(M, 128), _cdiv(N, 128), 4 * _cdiv(M, 4)
        st["x"] = _activations(gen, M, N, dev)
        code = lambda: torch.empty(M, N, dtype=torch.float8_e4m3fn, device=dev)  # noqa: E731
        scale = lambda *shape: torch.empty(shape, dtype=sdt, device=dev)         # noqa: E731
        st["out"] = {}
        if case["rows"]:
            st["out"].update(Xr=code(), sR=scale(words(Nb), ld))
        if case["cols"]:
            st["out"].update(Xc=code(), sC=scale(words(Mb), 4 * _cdiv(N, 4)))
        if case["blocks"]:
            st["out"].update(Xb=code(), sB=scale(Mb, words(Nb)), sBt=scale(Nb, words(Mb)))
        return st

    I, K, G, M = case["I"], case["K"], case["G"], _rows(case)
    nI, nK, nM = 2 * I // 128, _cdiv(K, 128), _cdiv(M, 128)
    x = _activations(gen, M, K, dev)
    if case["layout"] == "grouped":
        sizes = _groups(case, seed)
        starts = [0]
        for n in sizes:
            starts.append(starts[-1] + 128 * _cdiv(n, 128))
        index = [-1] * M
        for g, n in enumerate(sizes):
            index[starts[g]:starts[g] + n] = [g] * n
        st["m_indices"] = torch.tensor(index, dtype=torch.int32, device=dev)
        st["k_offsets"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        st["counts"] = torch.tensor(sizes, device=dev)
        st["most"] = max(sizes)                       # rows of the largest group
        x[st["m_indices"] < 0] = 0
    w = torch.randn(G, 2 * I, K, generator=gen, device=dev) * (1.0 / math.sqrt(K))
    st["W"], sw = _cast(w, 128, 128, scales)
    del w
    if case["op"] == "ffn_fwd":
        st["X"], sx = _cast(x.float(), 1, 128, scales)
        st["sX"] = _lay_rows(sx, scales)
        st["sW"] = _lay_last(sw, scales)
        st["h"] = torch.zeros(M, I, dtype=torch.bfloat16, device=dev)
        st["gu"] = torch.zeros(M, 2 * I, dtype=torch.bfloat16, device=dev) if case["save"] else None
    else:
        st["Xb"], sxb = _cast(x.float(), 128, 128, scales)      # from the forward pass: X in blocks for dW
        st["sXb"] = _lay_last(sxb.t(), scales)                  # [ceil(K/128), ceil(M/128)]
        st["sWt"] = _lay_last(sw.transpose(1, 2), scales)       # [G, ceil(K/128), 2I/128]
        st["gu"] = torch.randn(M, 2 * I, generator=gen, device=dev).to(torch.bfloat16)
        st["dh"] = (0.02 * torch.randn(M, I, generator=gen, device=dev)).to(torch.bfloat16)
        st["q_rows"] = torch.empty(M, 2 * I, dtype=torch.float8_e4m3fn, device=dev)
        st["s_rows"] = torch.empty(words(nI), 4 * _cdiv(M, 4), dtype=sdt, device=dev)
        st["q_cols"] = torch.empty(M, 2 * I, dtype=torch.float8_e4m3fn, device=dev)
        st["s_cols"] = torch.empty(words(nM), 2 * I, dtype=sdt, device=dev)
        st["dx"] = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
        st["dw"] = torch.zeros(G, 2 * I, K, dtype=torch.bfloat16, device=dev)
    if case["layout"] == "dense":
        for k in ("W", "sW", "sWt", "dw"):
            if k in st:
                st[k] = st[k][0]
    return st


# ---------------------------------------------------------------------------------------- the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"dropout": _own_dropout, "cast": _own_cast, "ffn_fwd": _own_fwd, "ffn_bwd": _own_bwd}[op](state)
    return {"dropout": _plain_dropout, "cast": _plain_cast, "ffn_fwd": _plain_fwd, "ffn_bwd": _plain_bwd}[op](state)


def _own_dropout(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    return dg.dg_dropout(st["x"], st["y"], st["rng_dev"], st["case"]["p"], R=st["r"])


def _own_cast(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    (dg.dg_cast_fp8_ue8m0 if st["case"]["scales"] == "ue8m0" else dg.dg_cast_fp8)(st["x"], **st["out"])
    return st["out"]


def _own_fwd(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    case = st["case"]
    rng = st["rng_dev"] if case["p"] > 0 else None
    if case["layout"] == "dense":
        call = dg.dg_fp8_gemm_nt_swiglu_ue8m0 if case["scales"] == "ue8m0" else dg.dg_fp8_gemm_nt_swiglu
        call(st["X"], st["sX"], st["W"], st["sW"], st["h"], GU=st["gu"], rng=rng, p=case["p"])
    else:
        call = (dg.dg_fp8_grouped_contiguous_swiglu_ue8m0 if case["scales"] == "ue8m0"
                else dg.dg_fp8_grouped_contiguous_swiglu)
        call(st["X"], st["sX"], st["W"], st["sW"], st["m_indices"], st["h"], GU=st["gu"], rng=rng, p=case["p"])
    return {"h": st["h"], "gu": st["gu"]}


def _own_bwd(st):
    import moe_grouped_gemm_e4m3_gb300 as dg
    case = st["case"]
    ue, grouped = case["scales"] == "ue8m0", case["layout"] == "grouped"
    (dg.dg_swiglu_backward_fp8_ue8m0 if ue else dg.dg_swiglu_backward_fp8)(
        st["dh"], st["gu"], st["q_rows"], st["s_rows"], st["q_cols"], st["s_cols"],
        m_indices=st["m_indices"] if grouped else None, rng=st["rng_dev"] if case["p"] > 0 else None, p=case["p"])
    if grouped:
        (dg.dg_fp8_grouped_contiguous_nn_ue8m0 if ue else dg.dg_fp8_grouped_contiguous_nn)(
            st["q_rows"], st["s_rows"], st["W"], st["sWt"], st["m_indices"], st["dx"])
        (dg.dg_fp8_k_grouped_gemm_tn_contiguous_ue8m0 if ue else dg.dg_fp8_k_grouped_gemm_tn_contiguous)(
            st["q_cols"], st["s_cols"], st["Xb"], st["sXb"], st["k_offsets"], st["dw"])
    else:
        M, I, K = case["M"], case["I"], case["K"]
        (dg.dg_fp8_gemm_nn_ue8m0 if ue else dg.dg_fp8_gemm_nn)(
            st["q_rows"], st["s_rows"], st["W"], st["sWt"], st["dx"], M, K, 2 * I)
        (dg.dg_fp8_gemm_tn_ue8m0 if ue else dg.dg_fp8_gemm_tn)(
            st["q_cols"], st["s_cols"], st["Xb"], st["sXb"], st["dw"], 2 * I, K, M)
    return {"dx": st["dx"], "dw": st["dw"]}


def _plain_dropout(st):
    case = st["case"]
    y = _dropped(st["x"].float(), case["p"], st["rng"])
    if st["r"] is not None:
        y = st["r"].float() + y
    return y.to(st["x"].dtype)


def _plain_cast(st):
    case, x = st["case"], st["x"].float()
    scales, out = case["scales"], {}
    if case["rows"]:
        out["Xr"], s = _cast(x, 1, 128, scales)
        out["sR"] = _lay_rows(s, scales)
    if case["cols"]:
        out["Xc"], s = _cast(x, 128, 1, scales)
        out["sC"] = _lay_rows(s.t(), scales)
    if case["blocks"]:
        out["Xb"], s = _cast(x, 128, 128, scales)
        out["sB"], out["sBt"] = _lay_last(s, scales), _lay_last(s.t(), scales)
    return out


def _by_group(st, x):
    """x [M_total, ..] -> [G, most, ..], zeros past each group's rows, and the rows' places."""
    at = st["k_offsets"][:-1].long()[:, None] + torch.arange(max(1, st["most"]), device=x.device)
    live = torch.arange(max(1, st["most"]), device=x.device) < st["counts"][:, None]
    at = at.clamp_max(x.shape[0] - 1)
    return torch.where(live[..., None], x[at], torch.zeros((), dtype=x.dtype, device=x.device)), at, live


def _from_groups(y, at, live, M):
    out = torch.zeros(M, y.shape[-1], dtype=y.dtype, device=y.device)
    out[at[live]] = y[live]
    return out


def _plain_fwd(st):
    case = st["case"]
    scales, I, K, M = case["scales"], case["I"], case["K"], st["X"].shape[0]
    nK = _cdiv(K, 128)
    x = st["X"].float() * _spread(_unlay_rows(st["sX"], M, nK, scales), 1, 128, M, K)
    w = st["W"].float() * _spread(_unlay_last(st["sW"], nK, scales), 128, 128, 2 * I, K)
    if case["layout"] == "dense":
        d = x @ w.t()
    else:
        xg, at, live = _by_group(st, x)
        d = _from_groups(torch.bmm(xg, w.transpose(1, 2)), at, live, M)
    g, u = d[:, :I], d[:, I:]
    h = _dropped(g / (1.0 + torch.exp(-g)) * u, case["p"], st["rng"])
    return {"h": h.to(torch.bfloat16), "gu": d.to(torch.bfloat16) if case["save"] else None}


def _plain_bwd(st):
    case = st["case"]
    scales, I, K, M = case["scales"], case["I"], case["K"], st["gu"].shape[0]
    nI, nK, nM = 2 * I // 128, _cdiv(K, 128), _cdiv(M, 128)
    g, u = st["gu"][:, :I].float(), st["gu"][:, I:].float()
    t = _dropped(st["dh"].float(), case["p"], st["rng"])
    sig = 1.0 / (1.0 + torch.exp(-g))
    d = torch.cat([t * u * sig * (1.0 + g * (1.0 - sig)), t * g * sig], dim=1)
    if case["layout"] == "grouped":
        d = torch.where((st["m_indices"] >= 0)[:, None], d, torch.zeros_like(d))
    q, s = _cast(d, 1, 128, scales)
    rows = q.float() * _spread(s, 1, 128, M, 2 * I)
    q, s = _cast(d, 128, 1, scales)
    cols = q.float() * _spread(s, 128, 1, M, 2 * I)
    w = st["W"].float() * _spread(_unlay_last(st["sWt"], nI, scales).transpose(-1, -2), 128, 128, 2 * I, K)
    x = st["Xb"].float() * _spread(_unlay_last(st["sXb"], nM, scales).t(), 128, 128, M, K)
    if case["layout"] == "dense":
        dx, dw = rows @ w, cols.t() @ x
    else:
        rg, at, live = _by_group(st, rows)
        dx = _from_groups(torch.bmm(rg, w), at, live, M)
        dw = torch.bmm(_by_group(st, cols)[0].transpose(1, 2), _by_group(st, x)[0])
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


# ------------------------------------------------------------------- the definitions, in 64 bits

def _exact_decode(w, n):
    """Scales in 64 bits: FP32 ones as they are, packed words byte by byte."""
    if w.dtype != torch.int32:
        return w.double()
    b = torch.stack([(w >> (8 * j)) & 0xFF for j in range(4)], dim=-1).flatten(-2)
    return torch.pow(2.0, b[..., :n].double() - 127.0)


def _exact_at(s, rows, cols):
    """s at (rows // 128 or row, cols // 128 or column): by index, the last two axes."""
    return s[..., rows, :][..., cols]


def _exact_mask(shape, p, rng, device):
    """The kept elements, from the generator's definition with 16-bit limbs (no product passes 2^48)."""
    n = shape[0] * shape[1]
    i = torch.arange(_cdiv(n, 8), device=device)
    m16, m32 = 0xFFFF, 0xFFFFFFFF

    def mul(m, c):
        lo = m * (c & m16)
        hi = m * (c >> 16) + (lo >> 16)
        return hi >> 16, ((hi & m16) << 16) | (lo & m16)

    c = [i & m32, i >> 32, torch.full_like(i, rng[1] & m32), torch.full_like(i, (rng[1] >> 32) & m32)]
    for r in range(10):
        k0 = ((rng[0] & m32) + r * 0x9E3779B9) & m32
        k1 = (((rng[0] >> 32) & m32) + r * 0xBB67AE85) & m32
        h0, l0 = mul(0xD2511F53, c[0])
        h1, l1 = mul(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
    bits = torch.empty(i.numel(), 8, dtype=torch.int64, device=device)
    for j in range(4):
        bits[:, 2 * j], bits[:, 2 * j + 1] = c[j] & m16, c[j] >> 16
    drop = round(p * 65536)
    return (bits.flatten()[:n] >= drop).view(shape), 65536 / (65536 - drop)


def _exact_pow2(r):
    """The smallest power of two at or above r: the logarithm, put right where it was rounded across a whole number."""
    s = torch.pow(2.0, torch.round(torch.log2(r)))
    s = torch.where(s < r, 2 * s, s)
    return torch.where(s / 2 >= r, s / 2, s)


def _exact_cast(d, dim, scales):
    """d [M, N] in 64 bits through E4M3 with groups of 128 along `dim`, back in 64 bits."""
    out = torch.empty_like(d)
    for at in range(0, d.shape[dim], 128):
        part = d.narrow(dim, at, min(128, d.shape[dim] - at))
        top = part.abs().amax(dim=dim, keepdim=True)
        use = torch.where(top > 0, top.clamp_min(TINY), torch.full_like(top, LIMIT))
        s = _exact_pow2(use / LIMIT) if scales == "ue8m0" else use / LIMIT
        out.narrow(dim, at, part.shape[dim]).copy_((part / s).clamp(-LIMIT, LIMIT).to(torch.float8_e4m3fn).double() * s)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "cast":
        x = st["x"].double()
        out = {}
        if case["rows"]:                       # the codes' values; FP32 scales too (packed ones are whole numbers)
            out["Xr"], out["sR"] = _exact_codes(x, 1, case["scales"])
        if case["cols"]:
            out["Xc"], out["sC"] = _exact_codes(x, 0, case["scales"])
        if case["blocks"]:
            out["Xb"], out["sB"], out["sBt"] = _exact_blocks(x, case["scales"])
        return out
    if case["op"] == "dropout":
        x = st["x"].double()
        keep, scale = _exact_mask(x.shape, case["p"], st["rng"], x.device)
        y = torch.where(keep, x * scale, 0.0)
        return y if st["r"] is None else st["r"].double() + y
    scales, I, K, G = case["scales"], case["I"], case["K"], case["G"]
    M = st["gu"].shape[0] if st["gu"] is not None else st["X"].shape[0]
    dev = st["W"].device
    rows, feats, ks = torch.arange(M, device=dev), torch.arange(2 * I, device=dev), torch.arange(K, device=dev)
    W = st["W"].reshape(G, 2 * I, K)
    spans = [(0, M)] if case["layout"] == "dense" else [
        (a, a + n) for a, n in zip(st["k_offsets"].tolist(), st["counts"].tolist())]
    if case["op"] == "ffn_fwd":
        sx = _exact_decode(st["sX"].t(), _cdiv(K, 128))
        sw = _exact_decode(st["sW"].reshape((G,) + st["sW"].shape[-2:]), _cdiv(K, 128))
        d = torch.zeros(M, 2 * I, dtype=torch.float64, device=dev)
        for g, (a, b) in enumerate(spans):
            x = st["X"][a:b].double() * _exact_at(sx, rows[a:b], ks // 128)
            d[a:b] = x @ (W[g].double() * _exact_at(sw[g], feats // 128, ks // 128)).t()
        h = d[:, :I] * torch.sigmoid(d[:, :I]) * d[:, I:]
        if case["p"] > 0:
            keep, scale = _exact_mask(h.shape, case["p"], st["rng"], dev)
            h = torch.where(keep, h * scale, 0.0)
        return {"h": h, "gu": d if case["save"] else None}
    g, u, t = st["gu"][:, :I].double(), st["gu"][:, I:].double(), st["dh"].double()
    if case["p"] > 0:
        keep, scale = _exact_mask(t.shape, case["p"], st["rng"], dev)
        t = torch.where(keep, t * scale, 0.0)
    sig = torch.sigmoid(g)
    d = torch.cat([t * u * (sig + g * sig * (1 - sig)), t * (g * sig)], dim=1)
    if case["layout"] == "grouped":
        d[st["m_indices"] < 0] = 0.0
    by_row, by_col = _exact_cast(d, 1, scales), _exact_cast(d, 0, scales)
    sw = _exact_decode(st["sWt"].reshape((G,) + st["sWt"].shape[-2:]), 2 * I // 128).transpose(1, 2)
    sx = _exact_decode(st["sXb"], _cdiv(M, 128)).t()
    dx = torch.zeros(M, K, dtype=torch.float64, device=dev)
    dw = torch.zeros(G, 2 * I, K, dtype=torch.float64, device=dev)
    for k, (a, b) in enumerate(spans):
        dx[a:b] = by_row[a:b] @ (W[k].double() * _exact_at(sw[k], feats // 128, ks // 128))
        dw[k] = by_col[a:b].t() @ (st["Xb"][a:b].double() * _exact_at(sx, rows[a:b] // 128, ks // 128))
    return {"dx": dx, "dw": dw[0] if case["layout"] == "dense" else dw}


def _exact_codes(x, dim, scales):
    """The values of the codes of groups of 128 along `dim`, and the FP32 scales in the products' layout."""
    top = torch.stack([p.abs().amax(dim=dim) for p in x.split(128, dim)])          # [groups, other axis]
    top = torch.where(top > 0, top.clamp_min(TINY), torch.full_like(top, LIMIT))
    s = _exact_pow2(top / LIMIT) if scales == "ue8m0" else top / LIMIT
    at = torch.arange(x.shape[dim], device=x.device) // 128
    q = (x / (s[at].t() if dim == 1 else s[at])).clamp(-LIMIT, LIMIT).to(torch.float8_e4m3fn).double()
    return q, None if scales == "ue8m0" else _pad(s, s.shape[0], 4 * _cdiv(s.shape[1], 4))


def _exact_blocks(x, scales):
    """The values of the codes of 128x128 blocks and the FP32 scales, by blocks of rows and transposed."""
    top = torch.stack([torch.stack([b.abs().max() for b in r.split(128, 1)]) for r in x.split(128, 0)])
    top = torch.where(top > 0, top.clamp_min(TINY), torch.full_like(top, LIMIT))
    s = _exact_pow2(top / LIMIT) if scales == "ue8m0" else top / LIMIT
    at = [torch.arange(n, device=x.device) // 128 for n in x.shape]
    q = (x / _exact_at(s, at[0], at[1])).clamp(-LIMIT, LIMIT).to(torch.float8_e4m3fn).double()
    return (q, None, None) if scales == "ue8m0" else (q, s, s.t())
