"""The training operators together, as examples/expert_ffn_training.py uses them: one step's output and gradients
against the same layer in 64 bits, and a short training run.

Tolerance of the step: every product has two E4M3 operands, each rounded with a relative error of at most 2^-4
(3.6% in the mean square for values spread evenly over a binade, about 2.6% in practice), and five casts lie
on the way to dW1: independent errors add to 6-8% of the norm; 0.12 is asked for."""
import os
import sys

import pytest
import torch

import _train_ref as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _keep(rows, cols, p, rng):
    seed, offset = rng.tolist()
    mask = torch.from_numpy(R.keep_mask(0, rows * cols, p, seed, offset)).view(rows, cols).cuda()
    return mask.double() * R.keep_scale(p)


@pytest.mark.parametrize("scales", ["fp32", "ue8m0"])
def test_one_step_against_autograd(scales):
    import expert_ffn_training as ex
    sizes, K, I = (200, 0, 128, 1, 77), 256, 256
    rows = 128 * sum(R.cdiv(n, 128) for n in sizes)
    layer = ex.ExpertFFN(len(sizes), K, I, rows, scales, p_hidden=0.2, p_out=0.1, seed=3)
    m_indices, k_offsets = ex.route(sizes, rows)
    live = (m_indices >= 0)[:, None]
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(rows, K, generator=gen, device="cuda").bfloat16()      # padding rows hold values too
    dout = (torch.randn(rows, K, generator=gen, device="cuda") * 0.01).bfloat16() * live
    out = layer.forward(x, m_indices).clone()
    dx = layer.backward(dout, m_indices, k_offsets)

    xd = x.double().requires_grad_()
    w1, w2 = layer.w1.double().requires_grad_(), layer.w2.double().requires_grad_()
    kh, ko = _keep(rows, I, 0.2, layer.rng_hidden), _keep(rows, K, 0.1, layer.rng_out)
    want = torch.zeros(rows, K, dtype=torch.float64, device="cuda")
    for g, n in enumerate(sizes):
        s = slice(int(k_offsets[g]), int(k_offsets[g]) + n)
        gu = xd[s] @ w1[g].T
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:] * kh[s]
        want[s] = xd[s] + (h @ w2[g].T) * ko[s]
    want.backward(dout.double())
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())           # noqa: E731
    on = live[:, 0]
    assert rel(out[on] - x[on], (want - xd)[on].detach()) < 0.12
    assert rel(dx[on].float() - dout[on].float(), (xd.grad - dout.double())[on]) < 0.12
    assert rel(layer.dw1, w1.grad) < 0.12 and rel(layer.dw2, w2.grad) < 0.12
    assert (layer.dw1[1] == 0).all() and (layer.dw2[1] == 0).all()         # the expert without tokens
    assert ex.dg.dg_get_device_status() == 0


@pytest.mark.parametrize("scales", ["fp32", "ue8m0"])
def test_training_lowers_the_loss(scales):
    import expert_ffn_training as ex
    losses = ex.train(scales, steps=60)
    assert losses == ex.train(scales, steps=60), "a run is not reproducible"
    assert losses[-1] < 0.5 * losses[0], losses[::8]
