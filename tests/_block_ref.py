"""Plain 64-bit definitions of the operators around the experts' products, with the errors that FP32 arithmetic and one
rounding of each output allow. Written from the formulas, elementwise; independent of the library's own code.

Every `want` is a pair (value, bound): an output has to be within `bound` of `value`. The bounds count
  * one rounding of the output to its type, half a step (`half`: bf16 2^-8, e4m3 2^-4, FP32 2^-24 of the value);
  * the FP32 arithmetic in front of it: n operations on terms t cost at most n·2^-24·Σ|t|. A row's sum takes at most 32 terms
    one after another and ten levels of a tree, 2^-24·42 < 2^-18; the tensor cores' FP32 sums, which may truncate (2^-23 a step),
    of at most 2^5 steps a group and 2^7 groups or warps, stay below 2^-15.9 in the worst order; the bound for them is
    2^-16·Σ|t| where K is below 4096.
"""
import torch

LIMIT = 448.0
ROW_SUM = 2.0 ** -18


def half(dt):
    return torch.finfo(dt).eps / 2


def rounded(value, bound, dt):
    """A value and its bound after one rounding to dt (FP32 outputs too)."""
    return value, bound + half(dt) * (value.abs() + bound) + torch.finfo(dt).tiny


# ------------------------------------------------------------------------------------------- norms

def norm(X, W, B, w_after, gate, scale, eps, dt):
    x = X.double()
    M, N = x.shape
    out = {}
    r, er = x, torch.zeros_like(x)
    if B is not None:
        p, ep = B.double(), torch.zeros_like(x)
        if w_after is not None:
            ra = 1.0 / (p.square().mean(1) + eps).sqrt()
            out["rstd_after"] = (ra, ra * ROW_SUM)
            p = p * ra[:, None] * w_after.double()
            ep = p.abs() * (ROW_SUM + 2.0 ** -22)
        f = torch.ones(M, 1, dtype=torch.float64, device=x.device) if gate is None else gate.double()[:, None]
        f = f if scale is None else f * scale.double()
        t = f * p
        r = x + t
        er = f.abs() * ep + 2.0 ** -21 * t.abs() + 2.0 ** -24 * r.abs()
        out["R"] = rounded(r, er, dt)
    if W is not None:
        ms = r.square().mean(1) + eps
        rs = 1.0 / ms.sqrt()
        # of the mean square: its own sum, and R's errors
        ers = rs * (ROW_SUM + (r.abs() * er).mean(1) / ms)
        out["rstd"] = (rs, ers)
        y = r * rs[:, None] * W.double()
        ey = W.double().abs() * (rs[:, None] * er + r.abs() * ers[:, None]) + 2.0 ** -22 * y.abs()
        out["Y"] = rounded(y, ey, dt)
        out["y"] = (y, ey)
    return out


def cast_rows(y, ey, pow2):
    """Of rows known to within ey: the dequantised rows (value: y itself; bound: half a step of E4M3 under the largest scale
    possible, plus ey), and the scales (value, bound) [M, groups]; pow2 scales as a pair (lowest, highest)."""
    M, N = y.shape
    G = -(-N // 128)
    pad = torch.zeros(M, G * 128, dtype=torch.float64, device=y.device)
    pad[:, :N] = y.abs()
    pe = torch.zeros_like(pad)
    pe[:, :N] = ey
    top = pad.view(M, G, 128).amax(2)
    te = pe.view(M, G, 128).amax(2)
    if pow2:
        lo, hi = pow2_scale(top - te), pow2_scale(top + te)
        scales = (lo, hi)
        s = hi
    else:
        s = torch.where(top > 0, top.clamp_min(2.0 ** -100) / LIMIT, torch.ones_like(top))
        scales = (s, te / LIMIT + 2.0 ** -22 * s)
    full = s.repeat_interleave(128, 1)[:, :N]
    # half a step: 2^-4 of the value, or half of the smallest subnormal (2^-10) under the scale; products and divisions in FP32 too
    step = torch.maximum(half(torch.float8_e4m3fn) * y.abs(), 2.0 ** -10 * full)
    return (y, step * (1 + 2.0 ** -10) + 2 * ey + 2.0 ** -20 * y.abs()), scales


def pow2_scale(top):
    """The smallest power of two s with top / s <= 448 (1 for no group)."""
    m, e = torch.frexp(top.clamp_min(2.0 ** -100))
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=top.device), (e - 9 + (m > 0.875).to(e.dtype)).double())
    return torch.where(top > 0, s, torch.ones_like(s))


def norm_backward(dY, dR, R, rstd, W, B, rstd_after, w_after, gate, scale, dt):
    like = dY if dY is not None else dR
    M, N = like.shape
    dev = like.device
    zero = torch.zeros(M, N, dtype=torch.float64, device=dev)
    dr = zero if dR is None else dR.double()
    out = {}
    g, eg = dr, zero
    if dY is not None:
        dy, xh, w = dY.double(), R.double() * rstd.double()[:, None], W.double()
        rs = rstd.double()[:, None]
        gw = dy * w
        c = (gw * xh).mean(1, keepdim=True)
        ec = ROW_SUM * (gw * xh).abs().mean(1, keepdim=True)
        g = dr + rs * (gw - xh * c)
        size = dr.abs() + rs * (gw.abs() + xh.abs() * c.abs())
        eg = rs * xh.abs() * ec + 2.0 ** -21 * size
        out["dW"] = columns(dy * xh, 2.0 ** -22 * (dy * xh).abs(), M)
    out["dX"] = rounded(g, eg, dt)
    if B is None:
        return out
    one = torch.ones(1, dtype=torch.float64, device=dev)
    ga = one[:, None] if gate is None else gate.double()[:, None]
    sc = one if scale is None else scale.double()
    ra = one[:, None] if w_after is None else rstd_after.double()[:, None]
    bh = B.double() * ra
    p = bh if w_after is None else bh * w_after.double()
    # Σ scale·P·G as the sum of its parts
    parts = (sc * p).abs() * (dr.abs() if dY is None else dr.abs() + rs * (gw.abs() + xh.abs() * c.abs()))
    along = (sc * p * g).sum(1)
    ealong = ROW_SUM * 2 * parts.sum(1) + ((sc * p).abs() * eg).sum(1)
    if gate is not None:
        out["dgate"] = rounded(along, ealong, torch.float32)
    if scale is not None:
        out["dscale"] = columns(ga * p * g, (ga * p).abs() * eg + 2.0 ** -21 * (ga * p * g).abs(), M)
    q = ga * sc * g
    eq = (ga * sc).abs() * eg + 2.0 ** -22 * q.abs()
    if w_after is not None:
        out["dw_after"] = columns(q * bh, bh.abs() * eq + 2.0 ** -22 * (q * bh).abs(), M)
        wa = w_after.double()
        mean = ga[:, 0] * along / N
        emean = ga[:, 0].abs() * ealong / N + 2.0 ** -22 * mean.abs()
        db = ra * (q * wa - bh * mean[:, None])
        edb = ra * (wa.abs() * eq + bh.abs() * emean[:, None]) + 2.0 ** -21 * ra * ((q * wa).abs() + (bh * mean[:, None]).abs())
    else:
        db, edb = q, eq
    out["dB"] = rounded(db, edb, dt)
    return out


def columns(terms, bound, M):
    """Sums over the rows: at most M/152 + 1 terms one after another, a share of the partial rows, eight shares."""
    n = M / 152 + 1 + 1216 / 8 + 8
    return rounded(terms.sum(0), bound.sum(0) + n * 2.0 ** -24 * terms.abs().sum(0), torch.float32)


# ------------------------------------------------------------------------------------------ router

def scores(logits, kind):
    """In 64 bits; NaN and -inf score 0."""
    l = torch.where(torch.isnan(logits), -torch.inf, logits).double()
    if kind == "sigmoid":
        return torch.where(l > -torch.inf, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    top = l.amax(1, keepdim=True)
    e = torch.where(l > -torch.inf, torch.exp(l - torch.where(top > -torch.inf, top, 0.0)), 0.0)
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def route(logits, bias, k, kind, renorm, factor):
    """ids and weights, one token at a time."""
    s = scores(logits.float(), kind).cpu()
    l = logits.float().cpu()
    T, E = l.shape
    ids, w = torch.full((T, k), -1, dtype=torch.int32), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        key = l[t].double() if bias is None else s[t] + bias.double().cpu()
        out = torch.isnan(l[t]) | (l[t] == -torch.inf) | torch.isnan(key) | (key == -torch.inf)
        order = sorted((e for e in range(E) if not out[e]), key=lambda e: (-float(key[e]), e))[:k]
        for i, e in enumerate(order):
            ids[t, i], w[t, i] = e, s[t, e]
    if renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return ids, w * factor


# ----------------------------------------------------------------------------- products of few tokens

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def four_bit(q, s):
    """Values of E2M1 codes [.., K/2] (even k in the low half) with E8M0 bytes [.., K/32], in 64 bits."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=q.device)
    v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], dim=-1).flatten(-2)
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=q.device), s.double() - 127.0)
    scale = torch.where(s == 255, torch.nan, scale)
    return v * scale.repeat_interleave(32, -1)


def e8m0_words(w, n):
    """The values of n packed E8M0 codes along the last axis."""
    b = torch.stack([(w >> (8 * j)) & 0xFF for j in range(4)], dim=-1).flatten(-2)[..., :n]
    return torch.pow(torch.tensor(2.0, dtype=torch.float64, device=w.device), b.double() - 127.0)


def rows_value(A, sA, packed):
    M, K = A.shape
    n = -(-K // 128)
    s = e8m0_words(sA.t().contiguous(), n)[:M] if packed else sA.t()[:M].double()
    return A.view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 1)[:, :K]


def weight_value(q, s, form):
    """One expert's matrix [N, K] in 64 bits."""
    if form == "mxfp4":
        return four_bit(q, s)
    N, K = q.shape
    s = e8m0_words(s, -(-K // 128)) if form == "ue8m0" else s.double()
    return q.view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


ACC = 2.0 ** -16


def e4m3(v):
    return v.clamp(-LIMIT, LIMIT).float().to(torch.float8_e4m3fn).double()


def product(x, w, dt):
    y = x @ w.t()
    return rounded(y, ACC * (x.abs() @ w.abs().t()), dt)


def moe(A, sA, W1, sW1, W2, sW2, ids, weights, form, dt):
    """(value, bound) of the layer's output. The cast of h is part of the definition: where h's FP32 error can carry it over
    a border of E4M3 (or of a power-of-two scale), the neighbouring codes are allowed for."""
    x = rows_value(A, sA, form == "ue8m0")
    I = W1.shape[1] // 2
    N = W2.shape[1]
    y = torch.zeros(x.shape[0], N, dtype=torch.float64, device=x.device)
    ey = torch.zeros_like(y)
    for t, row in enumerate(ids.tolist()):
        for j, e in enumerate(row):
            if not 0 <= e < W1.shape[0]:
                continue
            w1, w2, c = weight_value(W1[e], sW1[e], form), weight_value(W2[e], sW2[e], form), float(weights[t, j])
            d, ed = w1 @ x[t], ACC * (w1.abs() @ x[t].abs())
            g, u = d[:I], d[I:]
            sg = torch.sigmoid(g)
            h = g * sg * u
            # |silu'| <= 1.1; the fast exponential and division: 2^-20
            eh = 1.1 * ed[:I] * (u.abs() + ed[I:]) + (g * sg).abs() * ed[I:] + 2.0 ** -20 * h.abs()
            hg, eg = h.view(-1, 128), eh.view(-1, 128)
            top, te = hg.abs().amax(1, keepdim=True), eg.amax(1, keepdim=True)
            if form == "ue8m0":
                options = [pow2_scale(top), pow2_scale(top - te), pow2_scale(top + te)]
            else:
                options = [torch.where(top > 0, top.clamp_min(2.0 ** -100) / LIMIT, torch.ones_like(top))]
            s = options[0]
            q = e4m3(hg / s) * s
            off = torch.zeros_like(q)
            for o in options:
                slack = eg / o + 2.0 ** -20 * (hg / o).abs() + (te / o) * (hg / o).abs() / LIMIT
                for v in (hg / o - slack, hg / o + slack):
                    off = torch.maximum(off, (e4m3(v) * o - q).abs())
            off = off + q.abs() * (te / top.clamp_min(2.0 ** -100) + 2.0 ** -21)
            q, off = q.flatten(), off.flatten()
            y[t] += c * (w2 @ q)
            ey[t] += abs(c) * (w2.abs() @ off + ACC * (w2.abs() @ q.abs()))
    return rounded(y, ey, dt)


def close(got, want, what=""):
    value, bound = want
    off = (got.double() - value).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / bound.clamp_min(1e-300)).max()):.3f} of its bound"
