"""The norms with several rows a CTA: rings of every depth, rows asked for ahead, the columns' sums over them, against the 64-bit
definition."""
import pytest
import torch

from test_gpu_norm import BF, F32, _backward, _check_backward, _check_forward, _data, _forward, _stats, dg  # noqa: F401

pytestmark = pytest.mark.gpu

# (type, rows, columns): four rows and more a CTA. The backward pass of a block's boundary has three rows in its ring for BF16 up to 8192
# columns and FP32 up to 1024, two or one for longer ones (BF16 12288 and 16384; FP32 5120 and 2112, 7168), none for 16384 in FP32 and for
# lengths that are no multiples of eight.
ROWS = [(BF, 4901, 264), (BF, 3043, 1024), (BF, 3047, 2048), (BF, 1370, 4096), (BF, 765, 7168), (BF, 641, 8192), (BF, 613, 8200), (BF, 620, 12288),
        (BF, 457, 16384), (BF, 3050, 1033), (F32, 4901, 136), (F32, 3043, 1024), (F32, 3801, 1032), (F32, 1831, 2112), (F32, 613, 5120), (F32, 619, 7168),
        (F32, 611, 12288), (F32, 459, 16384), (F32, 3050, 1033)]


@pytest.mark.parametrize("dt,M,N", ROWS)
def test_forward_of_many_rows(dg, dt, M, N):  # noqa: F811
    d = _data(M, N, dt)
    q = "fp32" if N % 16 == 0 else None
    _check_forward(_forward(dg, d, q), d, q)


@pytest.mark.parametrize("dt,M,N", ROWS)
def test_backward_of_many_rows(dg, dt, M, N):  # noqa: F811
    d = _data(M, N, dt)
    first = _backward(dg, d)
    _check_backward(first, d)
    try:
        dg.dg_set_num_sms(11)
        again = _backward(dg, d)
    finally:
        dg.dg_set_num_sms(0)
    assert all(torch.equal(first[n], again[n]) for n in first)


@pytest.mark.parametrize("dt,M,N", [(BF, 3043, 520), (F32, 1831, 2112), (BF, 3050, 1033)])
@pytest.mark.parametrize("dy,dr", [(True, False), (False, True)])
@pytest.mark.parametrize("after,gate,scale", [(True, False, True), (False, True, False), (False, False, False)])
def test_parts_of_many_rows(dg, dt, M, N, dy, dr, after, gate, scale):  # noqa: F811
    d = _data(M, N, dt, after=after, gate=gate, scale=scale)
    _check_backward(_backward(dg, d, dy, dr), d, dy, dr)


@pytest.mark.parametrize("dt,M,N", [(BF, 3043, 1024), (F32, 1831, 2112), (BF, 457, 16384), (F32, 459, 16384)])
def test_outputs_of_many_rows_may_be_inputs(dg, dt, M, N):  # noqa: F811
    """Rows ahead are asked for while this row's outputs are stored."""
    d = _data(M, N, dt)
    want, back = _forward(dg, d), _backward(dg, d)
    rs, ra = _stats(d)
    x, b = d["X"].clone(), d["B"].clone()
    dg.dg_residual_norm(x, d["W"], B=b, w_after=d["w_after"], gate=d["gate"], scale=d["scale"], R=x, Y=b, eps=1e-6)
    assert torch.equal(x, want["R"]) and torch.equal(b, want["Y"])
    for over, other in (("dY", "B"), ("X", "dR")):
        c = {n: t.clone() for n, t in d.items()}
        dg.dg_residual_norm_backward(c["dY"], c["X"], rs, c["W"], dR=c["dR"], B=c["B"], rstd_after=ra, w_after=c["w_after"], gate=c["gate"],
                                     scale=c["scale"], dX=c[over], dB=c[other])
        assert torch.equal(c[over], back["dX"]) and torch.equal(c[other], back["dB"])
