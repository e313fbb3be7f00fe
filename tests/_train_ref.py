"""Plain implementations of the training operators, in 64 bits (the casts in the IEEE FP32 steps that
define them), shared by their tests: the generator, the E4M3 casts, the gated projection and its gradient."""
from __future__ import annotations

import numpy as np
import torch

ALIGN = 4


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------- dropout

def philox(counter, key):
    """Philox4x32-10 of counters [.., 4] under a key of two words, from the published definition."""
    c = [np.asarray(counter)[..., j].astype(np.uint64) for j in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=-1)


def threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def keep_mask(start, n, p, seed, offset):
    """Elements start .. start + n - 1 (start a multiple of 8): True where kept."""
    assert start % 8 == 0
    i = np.arange(start // 8, start // 8 + cdiv(n, 8), dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    seed, offset = seed & (2**64 - 1), offset & (2**64 - 1)
    counter = np.stack([i & low, i >> np.uint64(32), np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)], -1)
    w = philox(counter, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], axis=-1).reshape(-1)[:n]
    return bits >= threshold(p)


def keep_scale(p):
    return 65536.0 / (65536.0 - threshold(p))


def rng_tensor(seed, offset, device="cuda"):
    u = np.array([seed % 2**64, offset % 2**64], np.uint64)
    return torch.from_numpy(u.view(np.int64).copy()).to(device)


# ------------------------------------------------------------------------------------- casts

def e4m3(x32):
    """FP32 values, clamped to ±448, to E4M3 codes (round to nearest even)."""
    t = torch.from_numpy(np.ascontiguousarray(np.clip(x32, np.float32(-448), np.float32(448)), dtype=np.float32))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_values(codes):
    t = codes if isinstance(codes, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(codes))
    return t.cpu().view(torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def scale_of(amax32, ue8m0):
    """(factor, scale as FP32 or UE8M0 code) of groups with these maxima, in FP32."""
    amax = np.asarray(amax32, np.float32)
    a = np.maximum(amax, np.float32(2.0 ** -100))
    zero = amax == 0
    with np.errstate(all="ignore"):
        if not ue8m0:
            return (np.where(zero, np.float32(1), np.float32(448) / a).astype(np.float32),
                    np.where(zero, np.float32(1), a / np.float32(448)).astype(np.float32))
        m, e = np.frexp(np.where(np.isinf(a), np.float32(1), a))
        code = e - 9 + (m > 0.875) + 127
        code = np.where(zero, 127, code)
        factor = np.ldexp(np.float32(1), 127 - code).astype(np.float32)
        factor = np.where(np.isinf(amax), np.float32(0), factor)
        return factor, np.where(np.isinf(amax), 255, code).astype(np.uint8)


def cast_groups(x32, gr, gc, ue8m0):
    """Codes [M, N] and scales [ceil(M/gr), ceil(N/gc)] of gr x gc groups of x [M, N] (FP32)."""
    M, N = x32.shape
    Mb, Nb = cdiv(M, gr), cdiv(N, gc)
    pad = np.zeros((Mb * gr, Nb * gc), np.float32)
    pad[:M, :N] = np.abs(x32)
    top = np.fmax.reduce(np.nan_to_num(pad, nan=0.0, posinf=np.inf).reshape(Mb, gr, Nb, gc), axis=(1, 3))
    f, s = scale_of(top, ue8m0)
    spread = np.repeat(np.repeat(f, gr, 0), gc, 1)[:M, :N]
    with np.errstate(all="ignore"):
        return e4m3(x32 * spread), s


def pack(codes):
    """UE8M0 codes [.., n] -> int32 words [.., ceil(n/4)], unused bytes 127."""
    n = codes.shape[-1]
    full = np.full(codes.shape[:-1] + (4 * cdiv(n, 4),), 127, np.uint8)
    full[..., :n] = codes
    return np.ascontiguousarray(full).view("<i4")


def lay_lines(s, ue8m0):
    """Scales [lines, kb] -> the layout [kb][align4(lines)] (packed: words), filler past the lines."""
    lines, n = s.shape
    ld = ALIGN * cdiv(lines, ALIGN)
    if ue8m0:
        full = np.full((ld, n), 127, np.uint8)
        full[:lines] = s
        return np.ascontiguousarray(pack(full).T)
    full = np.zeros((ld, n), np.float32)
    full[:lines] = s
    return np.ascontiguousarray(full.T)


def lay_last(s, ue8m0):
    return pack(s) if ue8m0 else np.ascontiguousarray(s)


def unlay_lines(t, lines, n):
    """Device scales [kb or words][align4(lines)] -> [lines, n] in 64 bits."""
    a = t.cpu().numpy()
    if a.dtype == np.int32:
        b = np.ascontiguousarray(a.T).view(np.uint8)[:lines, :n]
        return np.where(b == 255, np.nan, np.ldexp(1.0, b.astype(np.int64) - 127))
    return a.T[:lines].astype(np.float64)


def unlay_last(t, n):
    a = t.cpu().numpy()
    if a.dtype == np.int32:
        b = np.ascontiguousarray(a).view(np.uint8)[..., :n]
        return np.where(b == 255, np.nan, np.ldexp(1.0, b.astype(np.int64) - 127))
    return a.astype(np.float64)


def spread(s, gr, gc, M, N):
    return np.repeat(np.repeat(s, gr, -2)[..., :M, :], gc, -1)[..., :N]


# ------------------------------------------------------------------------------------- the gate

def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def gate(g, u):
    return g * sigmoid(g) * u


def gate_grad(g, u, t):
    s = sigmoid(g)
    return t * u * s * (1.0 + g * (1.0 - s)), t * g * s


def bf16(x):
    """64-bit values rounded to BF16, as FP32."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).to(torch.float32).numpy()


def to_dev_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).cuda()
