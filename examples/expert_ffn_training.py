"""Trains the experts of one mixture-of-experts feed-forward layer in FP8, every operator through libdg.

    y = x + dropout(W2 · dropout(silu(Wg x) · (Wu x)))        for the expert of each token

The tokens of each expert stand together, padded to 128 rows (the contiguous layout). One step casts the activations and the
weights to E4M3, runs both projections, the loss and the whole backward pass, and updates FP32 master weights.
No activation crosses to BF16 twice, no transposed copy of anything is made: each operand is stored once per
contraction it takes part in, in its own order.

    python examples/expert_ffn_training.py [--scales fp32|ue8m0] [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_e4m3_gb300 as dg  # noqa: E402


def cdiv(a, b):
    return -(-a // b)


class ExpertFFN:
    """The experts' weights, and buffers for `rows` rows of tokens (a multiple of 128)."""

    def __init__(self, experts, features, hidden, rows, scales="fp32", p_hidden=0.1, p_out=0.1, seed=0):
        assert rows % 128 == 0 and hidden % 128 == 0 and features % 128 == 0
        self.G, self.K, self.I, self.M, self.scales = experts, features, hidden, rows, scales
        self.p_hidden, self.p_out = p_hidden, p_out
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w1 = torch.randn(experts, 2 * hidden, features, generator=gen, device="cuda") * features ** -0.5
        self.w2 = torch.randn(experts, features, hidden, generator=gen, device="cuda") * hidden ** -0.5
        # {seed, offset}: the hidden units' and the output's masks come from two offsets, moved on every step
        self.rng_hidden = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")
        self.rng_out = torch.tensor([seed, 1], dtype=torch.int64, device="cuda")
        self.x8, self.h8, self.dy8, self.dgu8 = (self._forms(rows, n) for n in (features, hidden, features, 2 * hidden))
        self.w1_8, self.w2_8 = self._weights(2 * hidden, features), self._weights(features, hidden)
        bf = lambda n: torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.gu, self.h, self.y, self.out = bf(2 * hidden), bf(hidden), bf(features), bf(features)
        self.dy, self.dh, self.dx = bf(features), bf(hidden), bf(features)
        self.dw1, self.dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)

    def _fn(self, name, f32=False):
        return getattr(dg, name + ("_ue8m0" if self.scales == "ue8m0" else "") + ("_f32" if f32 else ""))

    def _words(self, n):
        return cdiv(n, 4) if self.scales == "ue8m0" else n

    def _scale(self, *shape):
        return torch.zeros(shape, dtype=torch.int32 if self.scales == "ue8m0" else torch.float32, device="cuda")

    def _forms(self, M, N):
        """Codes and scales of a matrix in each of its three forms."""
        code = lambda: torch.zeros(M, N, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
        m, n = M // 128, N // 128
        return dict(Xr=code(), sR=self._scale(self._words(n), M), Xc=code(), sC=self._scale(self._words(m), N),
                    Xb=code(), sBt=self._scale(n, self._words(m)))

    def _weights(self, N, K):
        return dict(Xb=torch.zeros(self.G, N, K, dtype=torch.float8_e4m3fn, device="cuda"),
                    sB=self._scale(self.G, N // 128, self._words(K // 128)), sBt=self._scale(self.G, K // 128, self._words(N // 128)))

    def forward(self, x, m_indices):
        cast, x8, h8, w1, w2 = self._fn("dg_cast_fp8"), self.x8, self.h8, self.w1_8, self.w2_8
        cast(self.w1.bfloat16(), **w1)                       # blocks: scales for the forward and the backward product
        cast(self.w2.bfloat16(), **w2)
        cast(x, Xr=x8["Xr"], sR=x8["sR"], Xb=x8["Xb"], sBt=x8["sBt"], m_indices=m_indices)
        self._fn("dg_fp8_grouped_contiguous_swiglu")(x8["Xr"], x8["sR"], w1["Xb"], w1["sB"], m_indices, self.h, GU=self.gu,
                                                     rng=self.rng_hidden, p=self.p_hidden)
        cast(self.h, Xr=h8["Xr"], sR=h8["sR"], m_indices=m_indices)
        self._fn("dg_fp8_grouped_contiguous")(h8["Xr"], h8["sR"], w2["Xb"], w2["sB"], m_indices, self.y)
        return dg.dg_dropout(self.y, self.out, self.rng_out, self.p_out, R=x)

    def backward(self, dout, m_indices, k_offsets):
        """From the output's gradient (zero in padding rows): dx, and dw1 and dw2 in FP32."""
        dy8, dgu8, h8, x8, w1, w2 = self.dy8, self.dgu8, self.h8, self.x8, self.w1_8, self.w2_8
        dg.dg_dropout(dout, self.dy, self.rng_out, self.p_out)
        self._fn("dg_cast_fp8")(self.dy, Xr=dy8["Xr"], sR=dy8["sR"], Xc=dy8["Xc"], sC=dy8["sC"], m_indices=m_indices)
        nn, kg = self._fn("dg_fp8_grouped_contiguous_nn"), self._fn("dg_fp8_k_grouped_gemm_tn_contiguous", f32=True)
        nn(dy8["Xr"], dy8["sR"], w2["Xb"], w2["sBt"], m_indices, self.dh)
        self._fn("dg_swiglu_backward_fp8")(self.dh, self.gu, dgu8["Xr"], dgu8["sR"], dgu8["Xc"], dgu8["sC"], Hb=h8["Xb"],
                                           sHb=h8["sBt"], m_indices=m_indices, rng=self.rng_hidden, p=self.p_hidden)
        nn(dgu8["Xr"], dgu8["sR"], w1["Xb"], w1["sBt"], m_indices, self.dx)
        kg(dgu8["Xc"], dgu8["sC"], x8["Xb"], x8["sBt"], k_offsets, self.dw1)
        kg(dy8["Xc"], dy8["sC"], h8["Xb"], h8["sBt"], k_offsets, self.dw2)
        return self.dx + dout

    def update(self, lr):
        self.w1 -= lr * self.dw1
        self.w2 -= lr * self.dw2
        for rng in (self.rng_hidden, self.rng_out):          # new masks in the next step
            rng[1] += 2


def route(sizes, rows):
    """m_indices and k_offsets of experts with these many tokens each, in buffers of `rows` rows."""
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + 128 * cdiv(n, 128))
    assert starts[-1] <= rows
    index = torch.full((rows,), -1, dtype=torch.int32)
    for g, n in enumerate(sizes):
        index[starts[g]:starts[g] + n] = g
    return index.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda")


def train(scales="fp32", steps=60, sizes=(300, 0, 128, 85), features=256, hidden=384, lr=0.2, seed=0):
    """Fits a fixed random map; returns the loss of each step."""
    rows = 128 * sum(cdiv(n, 128) for n in sizes)
    layer = ExpertFFN(len(sizes), features, hidden, rows, scales, seed=seed)
    m_indices, k_offsets = route(sizes, rows)
    live = (m_indices >= 0)[:, None]
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(rows, features, generator=gen, device="cuda").bfloat16() * live
    target = (x.float() + 0.5 * x.float().roll(1, 1)) * live
    losses = []
    for _ in range(steps):
        out = layer.forward(x, m_indices)
        err = (out.float() - target) * live
        losses.append(float(err.square().sum() / live.sum() / features))
        layer.backward((2 * err / live.sum()).bfloat16(), m_indices, k_offsets)
        layer.update(lr)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--scales", choices=("fp32", "ue8m0"), default="fp32")
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    got = train(a.scales, a.steps)
    print("loss by step:", " ".join("%.4f" % v for v in got[::max(1, len(got) // 10)]), "last %.4f" % got[-1])
