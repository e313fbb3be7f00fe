"""Dropout from the counter-based generator with the residual sum: every bit against the plain implementation
(FP32 product, FP32 sum, one rounding), over lengths, alignments, types, streams and captured graphs."""
import numpy as np
import pytest
import torch

import _train_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield m
    assert m.dg_get_device_status() == 0


DTYPES = [torch.bfloat16, torch.float32]
SEED, OFFSET = 0x9E3779B97F4A7C15, 0x123456789


def _want(x, r, p, seed=SEED, offset=OFFSET, start=0):
    keep = torch.from_numpy(R.keep_mask(start, x.numel(), p, seed, offset)).view(x.shape)
    scale = torch.tensor(R.keep_scale(p), dtype=torch.float32)
    y = torch.where(keep, x.cpu().float() * scale, torch.zeros(()))
    return (y if r is None else r.cpu().float() + y).to(x.dtype)


def _data(n, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g).to(dt).cuda()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 4096, 100003])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9999])
def test_matches_definition(dg, dt, n, residual, p):
    x, r = _data(n, dt), _data(n, dt, 1) if residual else None
    y = torch.full((n + 8,), 77.0, dtype=dt, device="cuda")     # the elements past n must stay
    dg.dg_dropout(x, y[:n], R.rng_tensor(SEED, OFFSET), p, R=r)
    assert torch.equal(y[:n].cpu(), _want(x, r, p))
    assert (y[n:] == 77).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_any_alignment(dg, dt, shift):
    n = 1000
    x, r = _data(n + shift, dt)[shift:], _data(n, dt, 1)
    y = torch.empty(n + 1, dtype=dt, device="cuda")[1:]
    dg.dg_dropout(x, y, R.rng_tensor(SEED, OFFSET), 0.25, R=r)
    assert torch.equal(y.cpu(), _want(x, r, 0.25))


@pytest.mark.parametrize("dt", DTYPES)
def test_in_place_and_backward(dg, dt):
    rng = R.rng_tensor(SEED, OFFSET)
    x, r = _data(5000, dt), _data(5000, dt, 1)
    want = _want(x, r, 0.3)
    y = r.clone()
    dg.dg_dropout(x, y, rng, 0.3, R=y)                      # onto the residual
    assert torch.equal(y.cpu(), want)
    z = x.clone()
    dg.dg_dropout(z, z, rng, 0.3)                           # onto itself
    assert torch.equal(z.cpu(), _want(x, None, 0.3))
    ones = torch.ones(5000, dtype=dt, device="cuda")        # the gradient: the same mask, by itself
    d = torch.empty_like(ones)
    dg.dg_dropout(ones, d, rng, 0.3)
    assert torch.equal(d != 0, torch.from_numpy(R.keep_mask(0, 5000, 0.3, SEED, OFFSET)).cuda())


def test_dropped_values_are_zero_whatever_they_were(dg):
    x = _data(4096, torch.float32)
    x[::3], x[1::3] = float("nan"), float("inf")
    y = torch.empty_like(x)
    dg.dg_dropout(x, y, R.rng_tensor(5, 6), 0.5)
    keep = torch.from_numpy(R.keep_mask(0, 4096, 0.5, 5, 6))
    y = y.cpu()
    assert (y[~keep] == 0).all()
    assert torch.isnan(y[::3][keep[::3]]).all() and torch.isinf(y[1::3][keep[1::3]]).all()


def test_no_probability_needs_no_generator(dg):
    x = _data(1001, torch.bfloat16)
    y = torch.empty_like(x)
    dg.dg_dropout(x, y, None, 0.0)
    assert torch.equal(x, y)
    e = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    dg.dg_dropout(e, e, R.rng_tensor(1, 2), 0.5)


def test_past_32_bit_offsets(dg):
    """More than 2^32 elements: the counters and addresses of the last ones."""
    n = (1 << 32) + 1000
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = _data(2000, torch.bfloat16)
    start = n - 2000                                        # a multiple of 8, below 2^32
    x[start:] = tail
    dg.dg_dropout(x, x, R.rng_tensor(SEED, OFFSET), 0.4)
    assert torch.equal(x[start:].cpu(), _want(tail, None, 0.4, start=start))
    del x
    torch.cuda.empty_cache()


def test_other_stream_and_captured_graph(dg):
    rng, x = R.rng_tensor(3, 0), _data(10000, torch.bfloat16)
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dg.dg_dropout(x, y, rng, 0.2, stream=s)
    s.synchronize()
    assert torch.equal(y.cpu(), _want(x, None, 0.2, 3, 0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_dropout(x, y, rng, 0.2)
        rng[1] += 1                                         # the program moves the offset on
    for step in range(3):                                   # each replay draws another mask
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), _want(x, None, 0.2, 3, step))


def test_refusals(dg):
    x = _data(64, torch.bfloat16)
    y, rng = torch.empty_like(x), R.rng_tensor(1, 2)
    for p in (-0.1, 1.0, 2.0, float("nan"), 0.999999):      # the last rounds to 1 in 1/65536
        with pytest.raises(dg.DGError) as e:
            dg.dg_dropout(x, y, rng, p)
        assert e.value.status == dg.DG_ERR_INVALID_ARG
    with pytest.raises(dg.DGError):
        dg.dg_dropout(x, y, None, 0.1)
    with pytest.raises(dg.DGError):
        dg.dg_dropout(x[:32], x[8:40], rng, 0.1)            # a shifted overlap
    with pytest.raises(ValueError):
        dg.dg_dropout(x, y[:32], rng, 0.1)
    with pytest.raises(TypeError):
        dg.dg_dropout(x, y.float(), rng, 0.1)
    with pytest.raises(TypeError):
        dg.dg_dropout(x.half(), y.half(), rng, 0.1)
    with pytest.raises(ValueError):
        dg.dg_dropout(x[::2], y[::2], rng, 0.1)             # not contiguous
    with pytest.raises(ValueError):
        dg.dg_dropout(x, y, rng.cpu(), 0.1)
    with pytest.raises(TypeError):
        dg.dg_dropout(x, y, rng.int(), 0.1)
