"""The router's order of scores far below the row's largest, whose logits' distance to it is rounded before the exponential."""
import math

import numpy as np
import pytest
import torch

import _block_ref as R
from test_gpu_route import _route, dg  # noqa: F401

pytestmark = pytest.mark.gpu


def _token(top, near, E, row, rng):
    """Logits of a token with the largest `top` and two others one float apart about `near`, whose distances to it round away from
    each other, and the bias that puts the smaller of the two first by less than that."""
    l = np.float32(near) + np.arange(4000, dtype=np.float32) * np.spacing(np.float32(abs(near)))
    off = (l - np.float32(top)).astype(np.float64) - (l.astype(np.float64) - float(np.float32(top)))
    at = int(np.argmax(off[1:] - off[:-1]))          # rounded down, then up
    apart = float(off[at + 1] - off[at])
    low, high = l[at], l[at + 1]
    gap = (float(high) - float(low)) + float(rng.uniform(0.1, 0.9)) * apart      # the bias, in parts of the score
    logits = np.full(E, -np.inf, np.float32)
    logits[0] = top
    first = rng.random() < 0.5
    i, j = (2 * row + 1, 2 * row + 2) if first else (2 * row + 2, 2 * row + 1)
    logits[i], logits[j] = low, high
    return logits, i, gap * math.exp(float(low) - float(np.float32(top)))


@pytest.mark.parametrize("top,near", [(4.3217, -6.5), (12.345678, -6.0), (40.123456, -5.5), (70.75, -6.25), (0.3217, -70.0)])
def test_scores_far_below_the_largest(dg, top, near):  # noqa: F811
    E, T = 256, 127
    rng = np.random.default_rng(int(100 * top))
    bias = np.zeros(E, np.float32)
    logits = np.zeros((T, E), np.float32)
    for t in range(T):
        logits[t], i, b = _token(top * (1 + 0.001 * t), near + 0.003 * t, E, t, rng)
        bias[i] = b
    l, b = torch.from_numpy(logits).cuda(), torch.from_numpy(bias).cuda()
    for k in (2, 3):
        ids, _ = _route(dg, l, k, b, score="softmax", renormalize=False)
        want, _ = R.route(l, b, k, "softmax", False, 1.0)
        assert torch.equal(ids.cpu(), want), int((ids.cpu() != want).any(1).sum())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(14, 11), (256, 20), (512, 32)])
def test_sums_that_tie_in_64_bits(dg, E, k, dt, score):  # noqa: F811
    """Equal biases (they move in steps) of scores too small for FP64 to see beside them: the lowest index first, whatever FP32 knows
    of the scores by themselves."""
    g = torch.Generator().manual_seed(E)
    l = (12 * torch.randn(64, E, generator=g) - 30).to(dt).cuda()
    b = (torch.round(16 * torch.randn(E, generator=g)) / 16).cuda()
    for bias in (b, torch.full_like(b, 0.5), torch.zeros_like(b)):
        ids, _ = _route(dg, l, k, bias, score=score, renormalize=False)
        want, _ = R.route(l, bias, k, score, False, 1.0)
        assert torch.equal(ids.cpu(), want), int((ids.cpu() != want).any(1).sum())
