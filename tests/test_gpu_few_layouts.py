"""The experts' layer and the four-bit product at sizes whose layouts the other tests' sizes do not have: tables that leave little
shared memory, and units of two tiles of rows (what sizes of a few thousand rows launch), in every kernel that there is."""
import pytest
import torch

import _block_ref as R
import _few_plan as P
from test_gpu_few import _call, _check, _dense, _four, _gen, _layer, _rows, dg  # noqa: F401

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("form", ["", "ue8m0", "mxfp4"])
@pytest.mark.parametrize("T,N", [(32, 2448), (32, 4096), (33, 4096), (33, 4864)])
def test_all_experts_and_choices_there_can_be(dg, form, T, N):  # noqa: F811
    d = _layer(form, T, 32, 1024, 64, 128, N)
    y = _check(dg, d)
    try:
        dg.dg_set_num_sms(7)
        assert torch.equal(_call(dg, d), y)
    finally:
        dg.dg_set_num_sms(0)


# (form, tokens, choices, experts, K, I, N); K with ends inside a unit where the form has such kernels, N half a unit in the last block
TWO_TILES = [(form, T, *rest) for form in ("", "ue8m0") for T, rest in
             ((1, (3, 4, 752, 1024, 2448)), (3, (1, 4, 768, 1024, 2448)), (8, (1, 8, 656, 384, 2448)), (9, (1, 8, 768, 384, 2448)),
              (13, (2, 24, 656, 128, 2448)), (16, (2, 24, 768, 128, 2448)), (17, (1, 32, 3984, 128, 2448)), (32, (2, 32, 3968, 128, 2448)),
              (40, (1, 32, 3984, 128, 4096)))]
TWO_TILES += [("mxfp4", T, *rest) for T, rest in
              ((1, (8, 8, 256, 768, 2448)), (3, (2, 6, 256, 1024, 2448)), (8, (1, 8, 512, 768, 2448)), (9, (1, 8, 256, 768, 2448)),
               (13, (2, 24, 256, 256, 2448)), (16, (2, 24, 512, 256, 2448)))]
# several items a CTA in both products
TWO_TILES += [("", 8, 2, 16, 528, 768, 19504), ("ue8m0", 12, 2, 16, 528, 768, 19504), ("mxfp4", 12, 2, 16, 512, 768, 19504)]


def _is_of_two_tiles(form, T, k, E, K, I, N):
    return [p[0] for p in P.layer(T, k, E, K, I, N, form)] == [2, 2]


@pytest.mark.parametrize("form,T,k,E,K,I,N", TWO_TILES)
def test_units_of_two_tiles(dg, form, T, k, E, K, I, N):  # noqa: F811
    assert _is_of_two_tiles(form, T, k, E, K, I, N)
    d = _layer(form, T, k, E, K, I, N)
    y = _check(dg, d)
    try:
        for pdl, sms in ((True, 0), (False, 0), (None, 5)):
            dg.dg_set_pdl(pdl)
            dg.dg_set_num_sms(sms)
            assert torch.equal(_call(dg, d), y), (pdl, sms)
    finally:
        dg.dg_set_num_sms(0)
        dg.dg_set_pdl(None)
    if T > 2:       # no expert, one of them twice
        d["ids"][1] = -1
        d["ids"][T - 1] = int(d["ids"][T - 1, 0])
        assert bool((_check(dg, d)[1] == 0).all())


@pytest.mark.parametrize("form,T,k,E,K,I,N", [("", 16, 2, 24, 656, 128, 2448), ("", 32, 2, 32, 3984, 128, 2448), ("ue8m0", 32, 2, 32, 3984, 128, 2448),
                                              ("mxfp4", 13, 2, 24, 256, 256, 2448)])
def test_units_of_two_tiles_with_any_number_of_tokens(dg, form, T, k, E, K, I, N):  # noqa: F811
    """One expert with 1 to T tokens in any order, the rest through others, one token twice through the same."""
    assert _is_of_two_tiles(form, T, k, E, K, I, N)
    for count in sorted({1, 7, 8, 9, 13, 16, 17, 25, T} & set(range(1, T + 1))):
        d = _layer(form, T, k, E, K, I, N, seed=count)
        order = torch.randperm(T, generator=torch.Generator().manual_seed(count)).cuda()
        d["ids"][:, 0] = torch.where(order < count, 2, 0)
        d["ids"][:, 1] = torch.where(order % 3 == 0, -1, torch.where(order % 3 == 1, 3, d["ids"][:, 0]))
        _check(dg, d)


@pytest.mark.parametrize("M", [1, 7, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(2440, 2560), (9752, 256), (9736, 768), (29192, 256)])
def test_four_bit_product_of_two_tiles(dg, M, N, K):  # noqa: F811
    assert P.dense(M, N, K)[0] == 2
    g = _gen(M)
    A, sA = _rows(g, M, K)
    B, sB = _four(g, N, K)
    y = _dense(dg, A, sA, B, sB)
    R.close(y, R.product(R.rows_value(A, sA, False), R.four_bit(B, sB), torch.float32), "D")
    assert torch.equal(_dense(dg, A, sA, B, sB, f32=False), y.to(BF))
    try:
        dg.dg_set_num_sms(7)
        assert torch.equal(_dense(dg, A, sA, B, sB), y)
    finally:
        dg.dg_set_num_sms(0)
