"""The int8 products by the forms they are cut in, against 64-bit formulas."""
import pytest
import torch

from activation_sparse_gated_tma_b200 import twell as tw
from tests.test_gpu_int8 import BF16, F32, _operand, _product64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(5, 300, 256), (200, 300, 256), (700, 300, 256), (2500, 2600, 640), (2049, 5130, 1000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gated_product_of_up_channels_without_a_scale(M, N, K, dtype):
    # h = u ReLU(g): where u is NaN so is h, for any g, and an infinite u gives NaN where ReLU(g) is 0.
    x, xs = _operand(M, K, 1)
    wg, gs = _operand(N, K, 2)
    wu, us = _operand(N, K, 3)
    good = tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype)
    us[17], us[N - 1], us[40] = float("nan"), float("nan"), float("inf")
    h = tw.int8_gated(x, xs, wg, gs, wu, us, out_dtype=dtype)
    assert bool(h[:, 17].isnan().all()) and bool(h[:, N - 1].isnan().all())
    ref = _product64(x, xs, wg[40:41], gs[40:41]).clamp_min(0) * _product64(x, xs, wu[40:41], us[40:41])
    assert torch.equal(h[:, 40:41].isnan(), ref.isnan()) and bool(ref.isnan().any())
    assert torch.equal(h[:, 40:41].isinf(), ref.isinf())
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[[17, 40, N - 1]] = False
    assert torch.equal(h[:, keep], good[:, keep])
