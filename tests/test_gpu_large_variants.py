"""The variants that only large tensors reach: several counters a thread, several tiles a persistent CTA, one CTA a tile
in the backward pass. Bit for bit against the plain implementation, or against calls on parts of the same tensors."""
import numpy as np
import pytest
import torch

import _train_ref as R

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x1234567890ABCDEF, 5


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield m
    assert m.dg_get_device_status() == 0


def _holes(rows):
    """Row indices with padding in other places of every tile, and one tile of padding alone."""
    r = np.arange(rows)
    idx = np.where((r * 7 + r // 128 * 3) % 11 < 2, -1, r % 5).astype(np.int32)
    idx[256:384] = -1
    return idx


@pytest.mark.parametrize("dt,n,residual", [(torch.bfloat16, 5_300_011, True), (torch.bfloat16, 5_300_008, False),
                                           (torch.float32, 2_700_013, True), (torch.float32, 2_700_016, False)])
def test_dropout_of_many_elements(dg, dt, n, residual):
    gen = torch.Generator().manual_seed(3)
    x, r = (torch.randn(n, generator=gen).to(dt) for _ in range(2))
    keep = torch.from_numpy(R.keep_mask(0, n, 0.2, SEED, OFFSET))
    y = torch.where(keep, x.float() * torch.tensor(R.keep_scale(0.2), dtype=torch.float32), torch.zeros(()))
    want = (r.float() + y if residual else y).to(dt)
    got = torch.empty(n, dtype=dt, device="cuda")
    dg.dg_dropout(x.cuda(), got, R.rng_tensor(SEED, OFFSET), 0.2, R=r.cuda() if residual else None)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("ue", [False, True], ids=["fp32", "ue8m0"])
def test_cast_of_many_tiles(dg, ue):
    M, N = 4000, 4112                                       # 1056 tiles: more than twice the resident CTAs
    rng = np.random.default_rng(4)
    x = R.to_dev_bf16(rng.standard_normal((M, N)) * np.exp(rng.uniform(-6, 6, (M, 1))) * np.exp(rng.uniform(-3, 3, (1, N))))
    idx = _holes(M)
    x32 = np.where(idx[:, None] < 0, np.float32(0), x.float().cpu().numpy())
    sdt, w = (torch.int32, (lambda n: R.cdiv(n, 512))) if ue else (torch.float32, lambda n: R.cdiv(n, 128))
    code = lambda: torch.full((M, N), 0x55, dtype=torch.uint8, device="cuda")                      # noqa: E731
    scale = lambda *s: torch.full(s, 0x55555555, dtype=torch.int32, device="cuda").view(sdt)       # noqa: E731
    out = dict(Xr=code(), sR=scale(w(N), M), Xc=code(), sC=scale(w(M), N), Xb=code(), sB=scale(R.cdiv(M, 128), w(N)),
               sBt=scale(R.cdiv(N, 128), w(M)))
    (dg.dg_cast_fp8_ue8m0 if ue else dg.dg_cast_fp8)(x, m_indices=torch.from_numpy(idx).cuda(), **out)
    for name, (gr, gc) in (("Xr", (1, 128)), ("Xc", (128, 1)), ("Xb", (128, 128))):
        q, s = R.cast_groups(x32, gr, gc, ue)
        assert np.array_equal(out[name].cpu().numpy(), q), name
        lays = {"Xr": {"sR": lambda: R.lay_lines(s, ue)}, "Xc": {"sC": lambda: R.lay_lines(s.T, ue)},
                "Xb": {"sB": lambda: R.lay_last(s, ue), "sBt": lambda: R.lay_last(np.ascontiguousarray(s.T), ue)}}[name]
        for k, lay in lays.items():
            assert np.array_equal(out[k].cpu().numpy().view(np.int32), lay().view(np.int32)), k


@pytest.mark.parametrize("ue", [False, True], ids=["fp32", "ue8m0"])
@pytest.mark.parametrize("blocks", [False, True], ids=["gradients", "with_h"])
def test_backward_of_many_tiles(dg, ue, blocks):
    """369 tiles, more than two a CTA, against calls on 512 rows at a time, whose 36 tiles a cluster of CTAs shares each."""
    M, I, part = 5200, 1152, 512
    gen = torch.Generator(device="cuda").manual_seed(6)
    dh, gu = (torch.randn(M, n, generator=gen, device="cuda").bfloat16() for n in (I, 2 * I))
    idx = torch.from_numpy(_holes(M)).cuda()
    f = dg.dg_swiglu_backward_fp8_ue8m0 if ue else dg.dg_swiglu_backward_fp8
    sdt, w = (torch.int32, (lambda n: R.cdiv(n, 512))) if ue else (torch.float32, lambda n: R.cdiv(n, 128))

    def run(a, b):
        rows = b - a
        o = dict(dGUr=torch.zeros(rows, 2 * I, dtype=torch.uint8, device="cuda"), sR=torch.zeros(w(2 * I), 4 * R.cdiv(rows, 4), dtype=sdt, device="cuda"),
                 dGUc=torch.zeros(rows, 2 * I, dtype=torch.uint8, device="cuda"), sC=torch.zeros(w(rows), 2 * I, dtype=sdt, device="cuda"))
        if blocks:
            o.update(Hb=torch.zeros(rows, I, dtype=torch.uint8, device="cuda"), sHb=torch.zeros(I // 128, w(rows), dtype=sdt, device="cuda"))
        f(dh[a:b], gu[a:b], m_indices=idx[a:b], **o)
        return o

    got = run(0, M)
    parts = [run(a, min(a + part, M)) for a in range(0, M, part)]
    for k, v in got.items():
        want = torch.cat([p[k] for p in parts], dim=1 if k in ("sR", "sHb") else 0)
        assert torch.equal(v.view(torch.int8), want.view(torch.int8)), k
