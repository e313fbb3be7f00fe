"""The experts' layer and the four-bit product at sizes whose layouts the other tests' sizes do not have."""
import pytest
import torch

from test_gpu_few import _call, _check, _layer, dg  # noqa: F401

pytestmark = pytest.mark.gpu


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
