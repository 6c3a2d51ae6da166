"""A scale of a tensor that is NaN shows in every result that it scales."""
import pytest
import torch

from swin_window_attention_gb300 import capi

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_nan_scales(T):
    g = torch.Generator().manual_seed(T)
    x, w = (torch.randn(n, 160, generator=g).bfloat16().to(DEV) for n in (T, 72))
    xq, wq = capi.quantize_fp4(x, "nvfp4"), capi.quantize_fp4(w, "nvfp4")
    nan = torch.full((1,), float("nan"), device=DEV)
    assert torch.isfinite(capi.linear_fp4(xq, wq)).all()
    bad_x = capi.Fp4Tensor(xq.codes, xq.scales, nan, "nvfp4", xq.shape)
    bad_w = capi.Fp4Tensor(wq.codes, wq.scales, nan, "nvfp4", wq.shape)
    for y in (capi.linear_fp4(bad_x, wq), capi.linear_fp4(xq, bad_w), capi.linear_fp4(x, bad_w), capi.linear_fp4(x, wq, x_scale=nan)):
        assert torch.isnan(y).all()
    assert torch.isnan(capi.dequantize_fp4(bad_x)).all()
