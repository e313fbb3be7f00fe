"""E4M3 casts of BF16 matrices, all three forms: codes and scales bit for bit against the plain cast in
IEEE FP32, at sizes around the 128-element groups, and on groups that hold zeros, NaN, infinities, tiny
values and exact powers of two."""
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


def _outputs(G, M, N, ue, forms):
    sdt = torch.int32 if ue else torch.float32
    words = (lambda n: R.cdiv(n, 4)) if ue else (lambda n: n)
    Mb, Nb, lm, ln = R.cdiv(M, 128), R.cdiv(N, 128), 4 * R.cdiv(M, 4), 4 * R.cdiv(N, 4)
    code = lambda: torch.full((G, M, N), 0x55, dtype=torch.uint8, device="cuda")   # noqa: E731
    scale = lambda *s: torch.full((G,) + s, 0x55555555, dtype=torch.int32, device="cuda").view(sdt)  # noqa: E731
    out = {}
    if "rows" in forms:
        out.update(Xr=code(), sR=scale(words(Nb), lm))
    if "cols" in forms:
        out.update(Xc=code(), sC=scale(words(Mb), ln))
    if "blocks" in forms:
        out.update(Xb=code(), sB=scale(Mb, words(Nb)), sBt=scale(Nb, words(Mb)))
    if "nt" in forms:
        out.update(Xb=code(), sB=scale(Mb, words(Nb)))
    return out


def _want(x32, ue, forms):
    want = {}
    if "rows" in forms:
        q, s = R.cast_groups(x32, 1, 128, ue)
        want.update(Xr=q, sR=R.lay_lines(s, ue))
    if "cols" in forms:
        q, s = R.cast_groups(x32, 128, 1, ue)
        want.update(Xc=q, sC=R.lay_lines(s.T, ue))
    if "blocks" in forms or "nt" in forms:
        q, s = R.cast_groups(x32, 128, 128, ue)
        want.update(Xb=q, sB=R.lay_last(s, ue))
        if "blocks" in forms:
            want["sBt"] = R.lay_last(np.ascontiguousarray(s.T), ue)
    return want


def _same(got, want, what):
    got = got.cpu().numpy()
    if want.dtype == np.uint8:                       # NaN codes carry either sign
        nan = (want & 0x7F) == 0x7F
        assert ((got & 0x7F)[nan] == 0x7F).all(), what
        assert (got[~nan] == want[~nan]).all(), what
    else:
        assert np.array_equal(got.view(np.int32), want.view(np.int32)), what


def _check(dg, x, ue, forms, m_indices=None, x32=None):
    """x: device [M, N] or [G, M, N] BF16."""
    g = x.dim() == 3
    out = _outputs(x.shape[0] if g else 1, *x.shape[-2:], ue, forms)
    call = dg.dg_cast_fp8_ue8m0 if ue else dg.dg_cast_fp8
    call(x, m_indices=m_indices, **{k: v if g else v[0] for k, v in out.items()})
    torch.cuda.synchronize()
    mats = x.float().cpu().numpy() if x32 is None else x32
    for i, m in enumerate(mats if g else [mats]):
        for k, w in _want(m, ue, forms).items():
            _same(out[k][i], w, f"{k} of {tuple(x.shape)} group {i}")


def _random(M, N, seed=0):
    rng = np.random.default_rng(seed)
    return R.to_dev_bf16(rng.standard_normal((M, N)) * np.exp(rng.uniform(-8, 8, (M, 1))) * np.exp(rng.uniform(-3, 3, (1, N))))


@pytest.mark.parametrize("ue", [False, True])
@pytest.mark.parametrize("M,N", [(1, 16), (3, 128), (127, 144), (128, 128), (129, 272), (300, 1040), (640, 528), (5, 2064)])
def test_all_forms(dg, M, N, ue):
    _check(dg, _random(M, N), ue, ("rows", "cols", "blocks"))


@pytest.mark.parametrize("ue", [False, True])
@pytest.mark.parametrize("forms", [("rows",), ("cols",), ("blocks",), ("nt",), ("rows", "blocks"), ("rows", "cols")])
def test_each_form_alone(dg, forms, ue):
    _check(dg, _random(200, 400, 1), ue, forms)


@pytest.mark.parametrize("ue", [False, True])
def test_groups_of_matrices(dg, ue):
    _check(dg, torch.stack([_random(130, 144, s) for s in range(3)]), ue, ("rows", "cols", "blocks"))


@pytest.mark.parametrize("ue", [False, True])
def test_special_groups(dg, ue):
    x = np.zeros((256, 256), np.float32)
    x[0, :128] = 1e-40                        # BF16 subnormals, below the smallest group maximum
    x[1, 0], x[1, 1] = 2.0 ** -100, -2.0 ** -101
    x[2, :128] = 448.0                        # exactly a scale of one
    x[3, 0], x[3, 1] = 450.0, 3.0             # just past it
    x[4, 5] = np.nan
    x[4, 6] = 2.0
    x[5, 128:] = np.nan
    x[6, 130], x[6, 131] = np.inf, 1.0
    x[7, 0] = -np.inf
    x[8, 0], x[8, 1] = 3.3e38, 1.0            # near the largest value
    x[9, 0] = -0.0
    x[200, 200] = 1.75 * 2.0 ** 20
    t = torch.from_numpy(x).to(torch.bfloat16)
    _check(dg, t.cuda(), ue, ("rows", "cols", "blocks"), x32=t.float().numpy())


@pytest.mark.parametrize("ue", [False, True])
def test_padding_rows_count_as_zero(dg, ue):
    x = _random(384, 144, 2)
    idx = np.zeros(384, np.int32)
    idx[100:128], idx[256:384] = -1, -1       # the end of a block, and a whole block
    x[torch.from_numpy(idx < 0).cuda()] = float("nan")
    clean = np.where((idx < 0)[:, None], 0, x.float().cpu().numpy()).astype(np.float32)
    _check(dg, x, ue, ("rows", "cols", "blocks"), m_indices=torch.from_numpy(idx).cuda(), x32=clean)


@pytest.mark.parametrize("ue", [False, True])
def test_forms_feed_the_products(dg, ue):
    """Rows and blocks as A and B of the NT and NN products, columns and blocks as those of TN: the product of
    the dequantised operands, in 64 bits, within the products' FP32 accumulation (K + 8 roundings of 2^-24
    of the sum of magnitudes) and half a BF16 step (2^-8 of the value at most)."""
    M, N, K = 200, 144, 272
    a, b, c = _random(M, K, 3), _random(N, K, 4), _random(M, N, 5)
    sfx = "_ue8m0" if ue else ""
    call = getattr(dg, "dg_cast_fp8" + sfx)
    fa, fb, fc = _outputs(1, M, K, ue, ("rows", "blocks")), _outputs(1, N, K, ue, ("blocks",)), _outputs(1, M, N, ue, ("cols", "rows"))
    for f, x in ((fa, a), (fb, b), (fc, c)):
        call(x, **{k: v[0] for k, v in f.items()})
    nK, nM, nN = R.cdiv(K, 128), R.cdiv(M, 128), R.cdiv(N, 128)
    A = R.e4m3_values(fa["Xr"][0]) * R.spread(R.unlay_lines(fa["sR"][0], M, nK), 1, 128, M, K)
    Ab = R.e4m3_values(fa["Xb"][0]) * R.spread(R.unlay_last(fa["sB"][0], nK), 128, 128, M, K)
    B = R.e4m3_values(fb["Xb"][0]) * R.spread(R.unlay_last(fb["sB"][0], nK), 128, 128, N, K)
    C = R.e4m3_values(fc["Xr"][0]) * R.spread(R.unlay_lines(fc["sR"][0], M, nN), 1, 128, M, N)
    Cc = R.e4m3_values(fc["Xc"][0]) * R.spread(R.unlay_lines(fc["sC"][0], N, nM).T, 128, 1, M, N)
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    getattr(dg, "dg_fp8_gemm_nt" + sfx)(fa["Xr"][0], fa["sR"][0], fb["Xb"][0], fb["sB"][0], d)
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")      # C · B
    getattr(dg, "dg_fp8_gemm_nn" + sfx)(fc["Xr"][0], fc["sR"][0], fb["Xb"][0], fb["sBt"][0], dx, M, K, N)
    dw = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")      # Cᵀ · A, over 200 rows: no multiple of 16
    getattr(dg, "dg_fp8_gemm_tn" + sfx)(fc["Xc"][0], fc["sC"][0], fa["Xb"][0], fa["sBt"][0], dw, N, K, M)
    for got, x, y, k in ((d, A, B.T, K), (dx, C, B, N), (dw, Cc.T, Ab, M)):
        ref, size = x @ y, np.abs(x) @ np.abs(y)
        err = np.abs(got.double().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + (k + 8) * 2.0 ** -24 * size * 1.01).all()


def test_refusals(dg):
    x = _random(64, 128)
    q = torch.empty(64, 128, dtype=torch.uint8, device="cuda")
    s = torch.empty(1, 64, device="cuda")
    with pytest.raises(dg.DGError) as e:
        dg.dg_cast_fp8(x)                                        # no form asked for
    assert e.value.status == dg.DG_ERR_INVALID_ARG
    with pytest.raises(dg.DGError):
        dg.dg_cast_fp8(x, Xr=q)                                  # codes without scales
    with pytest.raises(dg.DGError):
        dg.dg_cast_fp8(x, sR=s)
    with pytest.raises(ValueError):
        dg.dg_cast_fp8(x, Xr=q, sR=s[:, :60])
    with pytest.raises(TypeError):
        dg.dg_cast_fp8(x.float(), Xr=q, sR=s)
    with pytest.raises(TypeError):
        dg.dg_cast_fp8_ue8m0(x, Xr=q, sR=s)                      # FP32 scales to the packed call
    y = _random(64, 120)
    with pytest.raises(dg.DGError) as e:
        dg.dg_cast_fp8(y, Xr=q[:, :120].contiguous(), sR=s)      # N % 16
    assert e.value.status == dg.DG_ERR_ALIGNMENT
    with pytest.raises(dg.DGError) as e:                         # misaligned X
        dg.dg_cast_fp8(torch.empty(64 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(64, 128), Xr=q, sR=s)
    assert e.value.status == dg.DG_ERR_ALIGNMENT
    g = torch.stack([x, x])
    with pytest.raises(dg.DGError):                              # m_indices with several matrices
        dg.dg_cast_fp8(g, Xr=torch.stack([q, q]), sR=torch.stack([s, s]), m_indices=torch.zeros(64, dtype=torch.int32, device="cuda"))
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    dg.dg_cast_fp8(e, Xr=q[:0], sR=s[:, :0])                     # an empty matrix: nothing to do
