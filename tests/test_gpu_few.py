"""The experts' layer for a few tokens and the product with four-bit weights, against the plain 64-bit definition
(tests/_block_ref.py) and the grouped calls' own chain, at sizes, choices and values where they can go wrong."""
import pytest
import torch

import _block_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
FORMS = ["", "ue8m0", "mxfp4"]


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_e4m3_gb300 as m
    m.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield m
    assert m.dg_get_device_status() == 0


def _cdiv(a, b):
    return -(-a // b)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(g, *shape):
    """E4M3 codes of normal values."""
    return (100 * torch.randn(*shape, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(g, packed, *shape, spread=0.5):
    if packed:
        return torch.randint(0, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int32) & 0x03030303 | 0x78787878
    return 2.0 ** -6 * torch.exp(spread * torch.randn(*shape, generator=g, device="cuda"))


def _rows(g, M, K, packed=False):
    n = _cdiv(K, 128)
    return _codes(g, M, K), _scales(g, packed, _cdiv(n, 4) if packed else n, 4 * _cdiv(M, 4))


def _four(g, *shape):
    """E2M1 codes [.., N, K/2] and E8M0 bytes [.., N, K/32] of scales between 2^-8 and 2^-4."""
    q = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), generator=g, device="cuda", dtype=torch.uint8)
    return q, torch.randint(119, 124, shape[:-1] + (shape[-1] // 32,), generator=g, device="cuda", dtype=torch.uint8)


def _weights(g, form, E, N, K):
    if form == "mxfp4":
        return _four(g, E, N, K)
    n = _cdiv(K, 128)
    return _codes(g, E, N, K), _scales(g, form == "ue8m0", E, _cdiv(N, 128), _cdiv(n, 4) if form == "ue8m0" else n) * (1 if form == "ue8m0" else 0.02)


def _layer(form, T, k, E, K, I, N, seed=0):
    g = _gen(seed)
    d = dict(form=form)
    d["A"], d["sA"] = _rows(g, T, K, form == "ue8m0")
    d["W1"], d["s1"] = _weights(g, form, E, 2 * I, K)
    d["W2"], d["s2"] = _weights(g, form, E, N, I)
    d["ids"] = torch.argsort(torch.rand(T, E, generator=g, device="cuda"), dim=1)[:, :k].to(torch.int32).contiguous()
    d["w"] = torch.rand(T, k, generator=g, device="cuda") + 0.1
    return d


def _call(dg, d, f32=True, **extra):
    name = "dg_fp8_moe_swiglu" + ("_" + d["form"] if d["form"] else "") + ("_f32" if f32 else "")
    T, N = d["A"].shape[0], d["W2"].shape[1]
    buf = torch.full((T * N + 8,), 7.0, device="cuda", dtype=F32 if f32 else BF)
    y = getattr(dg, name)(d["A"], d["sA"], d["W1"], d["s1"], d["W2"], d["s2"], d["ids"], d["w"], buf[:T * N].view(T, N), **extra)
    torch.cuda.synchronize()
    assert bool((buf[T * N:] == 7).all()), "written past the end"
    return y


def _check(dg, d):
    y = _call(dg, d)
    R.close(y, R.moe(d["A"], d["sA"], d["W1"], d["s1"], d["W2"], d["s2"], d["ids"], d["w"], d["form"], F32), "Y")
    assert torch.equal(_call(dg, d, f32=False), y.to(BF))
    return y


SIZES = [(1, 1, 1, 128, 128, 16), (1, 8, 32, 512, 256, 512), (2, 2, 4, 32, 128, 48), (3, 3, 5, 288, 384, 144), (5, 4, 16, 2080, 128, 2080),
         (7, 2, 3, 1056, 640, 272), (8, 2, 70, 1024, 128, 128), (9, 3, 8, 160, 256, 80), (16, 2, 6, 1568, 256, 320), (17, 2, 5, 256, 128, 112),
         (32, 4, 9, 544, 384, 160), (33, 2, 4, 384, 128, 64), (70, 3, 7, 128, 256, 32)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,k,E,K,I,N", SIZES)
def test_layer_sizes(dg, form, T, k, E, K, I, N):
    _check(dg, _layer(form, T, k, E, K, I, N))


@pytest.mark.parametrize("form", ["", "ue8m0"])
@pytest.mark.parametrize("K", [16, 48, 144, 2064])
def test_layer_of_odd_k(dg, form, K):
    _check(dg, _layer(form, 4, 2, 5, K, 128, 32))


@pytest.mark.parametrize("form", FORMS)
def test_choices(dg, form):
    """No expert, fewer of them, one twice, all tokens on one, the last expert alone."""
    for T in (6, 20, 40):
        d = _layer(form, T, 3, 11, 256, 128, 64, seed=T)
        ids = d["ids"]
        ids[0] = -1
        ids[1, 1:] = -1
        ids[2, 1] = ids[2, 0]
        ids[3] = 10
        y = _check(dg, d)
        assert bool((y[0] == 0).all())
        ids[:] = 4
        _check(dg, d)
        ids[:] = -1
        assert bool((_check(dg, d) == 0).all())
        ids[:, 0] = 10
        _check(dg, d)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,K,I", [(13, 512, 256), (13, 288, 128), (32, 512, 256), (32, 288, 128)])
def test_experts_of_any_number_of_tokens(dg, form, T, K, I):
    """One expert with 1 to T tokens in any order, the rest through others, one token twice through the same."""
    for count in sorted({1, 2, 7, 8, 9, 15, 16, 17, 24, 25, 31, T} & set(range(1, T + 1))):
        d = _layer(form, T, 2, 4, K, I, 48, seed=count)
        order = torch.randperm(T, generator=torch.Generator().manual_seed(count)).cuda()
        d["ids"][:, 0] = torch.where(order < count, 2, 0)
        d["ids"][:, 1] = torch.where(order % 3 == 0, -1, torch.where(order % 3 == 1, 3, d["ids"][:, 0]))
        _check(dg, d)


@pytest.mark.parametrize("form", FORMS)
def test_ids_out_of_range_are_flagged_and_count_as_none(dg, form):
    d = _layer(form, 5, 2, 4, 256, 128, 64)
    d["ids"][1, 0], d["ids"][3, 1] = 4, -2
    y = _call(dg, d)
    assert dg.dg_get_device_status() == dg.DG_DEV_BAD_GROUP_INDEX
    d["ids"][1, 0], d["ids"][3, 1] = -1, -1
    assert torch.equal(_call(dg, d), y) and dg.dg_get_device_status() == 0


@pytest.mark.parametrize("form", FORMS)
def test_a_nan_stays_with_its_tokens(dg, form):
    """A NaN in an expert's weights or scales reaches the tokens of that expert, one in a token's row that token."""
    for T in (5, 20):
        d = _layer(form, T, 1, 4, 256, 128, 64)
        d["ids"][:] = (torch.arange(T, device="cuda") % 3)[:, None]
        y = _check(dg, d)
        for name, at in (("W1", 3), ("W2", 1), ("s1", 1)):
            bad = {n: t.clone() if torch.is_tensor(t) else t for n, t in d.items()}
            if name == "W2" and form == "mxfp4":
                name = "s2"
            # 0x7F: E4M3's NaN; all ones: NaN as FP32, as packed codes and as a byte
            bad[name][at] = {torch.uint8: 0xFF if name[0] == "s" else 0x7F, torch.int32: -1, F32: float("nan")}[bad[name].dtype] if not (
                form == "mxfp4" and name[0] == "W") else bad[name][at]
            z = _call(dg, bad)
            hit = d["ids"][:, 0] == at
            assert torch.equal(z[~hit], y[~hit])
            if at == 1:
                assert bool(torch.isnan(z[hit]).all())
        bad = {**d, "A": d["A"].clone()}
        bad["A"][2, 7] = 0x7F
        z = _call(dg, bad)
        keep = torch.arange(T, device="cuda") != 2
        assert torch.equal(z[keep], y[keep]) and bool(torch.isnan(z[2]).all())


@pytest.mark.parametrize("form", ["", "ue8m0"])
def test_agrees_with_the_grouped_calls(dg, form):
    """The grouped calls' chain on the same weights: gather, gated product to FP8, down product, weighted sum in 64 bits."""
    T, k, E, K, I, N = 6, 2, 4, 512, 256, 384
    d = _layer(form, T, k, E, K, I, N)
    tail = "_ue8m0" if form else ""
    slots = [[] for _ in range(E)]
    for t, row in enumerate(d["ids"].tolist()):
        for j, e in enumerate(row):
            slots[e].append((t, j))
    rows = 128
    m = torch.tensor([len(s) for s in slots], dtype=torch.int32, device="cuda")
    A = torch.zeros(E, rows, K, dtype=torch.uint8, device="cuda")
    sA = torch.zeros(E, d["sA"].shape[0], rows, dtype=d["sA"].dtype, device="cuda")
    for e, s in enumerate(slots):
        for i, (t, _) in enumerate(s):
            A[e, i], sA[e, :, i] = d["A"][t], d["sA"][:, t]
    H = torch.zeros(E, rows, I, dtype=F32, device="cuda")
    getattr(dg, f"dg_fp8_grouped_masked_swiglu{tail}_f32")(A, sA, d["W1"], d["s1"], m, H)
    y = _call(dg, d)
    want, bound = R.moe(d["A"], d["sA"], d["W1"], d["s1"], d["W2"], d["s2"], d["ids"], d["w"], form, F32)
    total = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for e, s in enumerate(slots):
        w2 = R.weight_value(d["W2"][e], d["s2"][e], form)
        for i, (t, j) in enumerate(s):
            h = H[e, i].double().view(-1, 128)
            top = h.abs().amax(1, keepdim=True)
            sc = R.pow2_scale(top) if form else top / 448
            total[t] += float(d["w"][t, j]) * (w2 @ (R.e4m3(h / sc) * sc).flatten())
    assert bool(((total - want).abs() <= bound).all()) and bool(((y.double() - want).abs() <= bound).all())


def test_offsets_past_32_bits(dg):
    """Experts whose weights start behind the 2^31st and 2^32nd byte."""
    E, K, I, N = 160, 7168, 2048, 16
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    g = _gen(3)
    d = dict(form="", w=torch.ones(2, 2, device="cuda"))
    d["A"], d["sA"] = _rows(g, 2, K)
    d["W1"] = torch.zeros(E, 2 * I, K, dtype=torch.uint8, device="cuda")
    d["s1"] = _scales(g, False, E, 2 * I // 128, K // 128) * 0.02
    d["W2"], d["s2"] = _weights(g, "", E, N, I)
    d["ids"] = torch.tensor([[159, 74], [147, 0]], dtype=torch.int32, device="cuda")
    for e in (159, 74, 147, 0):
        d["W1"][e] = _codes(g, 2 * I, K)
    _check(dg, d)


@pytest.mark.parametrize("form", FORMS)
def test_same_bits_under_every_launch_setting(dg, form, monkeypatch):
    d = _layer(form, 12, 3, 9, 1056, 384, 272)
    y = _call(dg, d)
    before = dg.dg_get_pdl()
    try:
        for pdl, sms in ((True, 0), (False, 0), (None, 5), (None, 1)):
            dg.dg_set_pdl(pdl)
            dg.dg_set_num_sms(sms)
            assert torch.equal(_call(dg, d), y), (pdl, sms)
    finally:
        dg.dg_set_num_sms(0)
        dg.dg_set_pdl(before)
    need = dg.dg_fp8_moe_workspace(12, 3, 384)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    assert torch.equal(_call(dg, d, workspace=ws[:need]), y) and bool((ws[need:] == 0xA5).all())
    with pytest.raises(dg.DGError, match="workspace"):
        _call(dg, d, workspace=ws[:need - 16])
    args = [d[n] for n in ("A", "sA", "W1", "s1", "W2", "s2", "ids", "w")]
    assert dg._bind().moe(2 * FORMS.index(form) + 1, *args, torch.empty_like(y), None, None) == 0      # the short path takes it
    monkeypatch.setattr(dg, "_bind", lambda: dg._NoBind)
    assert torch.equal(_call(dg, d), y)


@pytest.mark.parametrize("form", FORMS)
def test_calls_at_once_and_one_behind_the_other(dg, form):
    ds = [_layer(form, 4, 2, 6, 512, 256, 256, seed=i) for i in range(3)]
    want = [_call(dg, d) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    name = "dg_fp8_moe_swiglu" + ("_" + form if form else "") + "_f32"
    for _ in range(4):
        got = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append(getattr(dg, name)(d["A"], d["sA"], d["W1"], d["s1"], d["W2"], d["s2"], d["ids"], d["w"], torch.empty_like(want[0])))
        for d in ds:        # back to back on one stream: each early start waits for what it needs
            got.append(getattr(dg, name)(d["A"], d["sA"], d["W1"], d["s1"], d["W2"], d["s2"], d["ids"], d["w"], torch.empty_like(want[0]),
                                         stream=streams[0]))
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert torch.equal(g, want[i % 3])


@pytest.mark.parametrize("form", FORMS)
def test_captured_and_replayed_with_other_choices(dg, form):
    d, other = _layer(form, 6, 2, 8, 512, 256, 128), _layer(form, 6, 2, 8, 512, 256, 128, seed=5)
    name = "dg_fp8_moe_swiglu" + ("_" + form if form else "") + "_f32"
    args = [d[n] for n in ("A", "sA", "W1", "s1", "W2", "s2", "ids", "w")]
    y = torch.empty(6, 128, device="cuda")
    getattr(dg, name)(*args, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        getattr(dg, name)(*args, y)
    for n in ("A", "sA", "ids", "w"):
        d[n].copy_(other[n])
    d["ids"][2] = -1
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, _call(dg, d))


# ------------------------------------------------------------------------------ four-bit weights

def _dense(dg, A, sA, B, sB, f32=True):
    M, N = A.shape[0], B.shape[0]
    buf = torch.full((M * N + 8,), 7.0, device="cuda", dtype=F32 if f32 else BF)
    y = (dg.dg_fp8_mxfp4_gemm_nt_f32 if f32 else dg.dg_fp8_mxfp4_gemm_nt)(A, sA, B, sB, buf[:M * N].view(M, N))
    torch.cuda.synchronize()
    assert bool((buf[M * N:] == 7).all())
    return y


@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 16, 256), (1, 2112, 7168 // 2), (2, 24, 96), (3, 200, 288), (5, 1000, 160), (8, 264, 1056),
                                   (9, 72, 2080), (16, 576, 512), (17, 104, 640), (31, 48, 128), (33, 88, 384), (100, 40, 1024)])
def test_four_bit_product(dg, M, N, K):
    g = _gen(M)
    A, sA = _rows(g, M, K)
    B, sB = _four(g, N, K)
    y = _dense(dg, A, sA, B, sB)
    R.close(y, R.product(R.rows_value(A, sA, False), R.four_bit(B, sB), F32), "D")
    assert torch.equal(_dense(dg, A, sA, B, sB, f32=False), y.to(BF))


def test_every_code_and_every_scale(dg):
    """One code a product: all sixteen codes under all scales that the FP32 sum can hold, NaN among them."""
    K = 32
    A = torch.zeros(1, K, dtype=torch.uint8, device="cuda")
    A[0, 5] = 0x38                                                     # 1.0
    sA = torch.ones(1, 4, device="cuda")
    B = torch.zeros(16 * 256, K // 2, dtype=torch.uint8, device="cuda")
    code = torch.arange(16, device="cuda").repeat_interleave(256)
    B[:, 2] = (code << 4).to(torch.uint8)                              # k = 5: the high half of byte 2
    sB = torch.arange(256, device="cuda").repeat(16).to(torch.uint8)[:, None].contiguous()
    got = _dense(dg, A, sA, B, sB)[0].double()
    want = R.four_bit(B, sB)[:, 5]
    want = torch.where(torch.isnan(want), want, want.float().double())      # 6·2^127 is past FP32
    assert bool(torch.isnan(got[sB[:, 0] == 255]).all())
    rest = sB[:, 0] != 255
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("N", [16, 5000])
@pytest.mark.parametrize("K", [32, 1056])
def test_four_bit_passes_follow_one_another(dg, N, K):
    """Many passes of 32 rows in one call, of one item a CTA and hardly any work, give the bits of a call for each pass."""
    M = 32 * 60 + 7
    g = _gen(11)
    A, _ = _rows(g, M, K)
    scales = _scales(g, False, _cdiv(K, 128), M)      # one a row and group, laid out for each call below
    B, sB = _four(g, N, K)

    def product(rows):
        n = rows.stop - rows.start
        s = torch.zeros(scales.shape[0], 4 * _cdiv(n, 4), device="cuda")
        s[:, :n] = scales[:, rows]
        D = torch.empty(n, N, device="cuda")
        dg.dg_fp8_mxfp4_gemm_nt_f32(A[rows], s, B, sB, D)
        return D

    want = torch.cat([product(slice(m, min(m + 32, M))) for m in range(0, M - 7, 32)])
    for _ in range(20):
        assert torch.equal(product(slice(0, M))[:M - 7], want)


def test_four_bit_launch_settings(dg, monkeypatch):
    g = _gen(1)
    A, sA = _rows(g, 11, 1120)
    B, sB = _four(g, 520, 1120)
    y = _dense(dg, A, sA, B, sB)
    try:
        for sms in (1, 7):
            dg.dg_set_num_sms(sms)
            assert torch.equal(_dense(dg, A, sA, B, sB), y)
    finally:
        dg.dg_set_num_sms(0)
    gr, out = torch.cuda.CUDAGraph(), torch.empty_like(y)
    with torch.cuda.graph(gr):
        dg.dg_fp8_mxfp4_gemm_nt_f32(A, sA, B, sB, out)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
    s = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    dg.dg_fp8_mxfp4_gemm_nt_f32(A, sA, B, sB, out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, y) and dg._bind().mxfp4(1, A, sA, B, sB, out, None) == 0
    monkeypatch.setattr(dg, "_bind", lambda: dg._NoBind)
    assert torch.equal(_dense(dg, A, sA, B, sB), y)
