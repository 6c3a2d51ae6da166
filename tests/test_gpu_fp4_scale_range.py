"""NVFP4 products whose two tensor scales multiply to something that fp32 does not hold, though the results do."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.linear_util import assert_within
from tests.test_gpu_fp4 import linear64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _values(q):
    return capi.dequantize_fp4(q, torch.float32).double().cpu()


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_small_scales(T, given):
    """Scales of 2^-65 each, results of some 2^-108. (A product that is flushed to zero would be wrong by all of it.)"""
    x, w = (_rand(T, T, 160) * 2.0 ** -56).bfloat16().to(DEV), (_rand(1, 72, 160) * 2.0 ** -56).bfloat16().to(DEV)
    wq = capi.quantize_fp4(w, "nvfp4")
    scale = torch.full((1,), 2.0 ** -65, device=DEV) if given else None
    xq = capi.quantize_fp4(x, "nvfp4", scale=scale)
    assert float(xq.tensor_scale) * float(wq.tensor_scale) < 2.0 ** -127
    ref, tol = linear64(_values(xq), _values(wq), None, "none", None)
    assert float(ref.abs().max()) > 2.0 ** -110 and float((tol / ref.abs().clamp_min(2.0 ** -115)).min()) < 2.0 ** -7
    for y in (capi.linear_fp4(x, wq, x_scale=scale), capi.linear_fp4(xq, wq)):
        assert_within("y", y.double() * 2.0 ** 108, ref * 2.0 ** 108, tol * 2.0 ** 108)


@pytest.mark.parametrize("T", [4, 40, 300])
def test_large_scales(T):
    """Scales of 2^71 and 2^61: results beyond fp32 are infinities, those within it are there, and a token or a channel of
    zeros gives the bias."""
    K, N = 128, 72
    x, w, b = _rand(T, T, K) * 2.0 ** 80, _rand(1, N, K) * 2.0 ** 70, _rand(2, N)
    x[1], w[6] = 0.0, 0.0
    x[2] *= 2.0 ** -16
    w[5] *= 2.0 ** -16
    x, w = x.bfloat16().to(DEV), w.bfloat16().to(DEV)
    wq, xq = capi.quantize_fp4(w, "nvfp4"), capi.quantize_fp4(x, "nvfp4")
    assert float(xq.tensor_scale.double() * wq.tensor_scale.double()) > 2.0 ** 129
    scale = xq.tensor_scale.clone()
    ref, tol = linear64(_values(xq), _values(wq), b, "none", None)
    fine = ref.abs() < 3e38
    assert fine[1].all() and fine[:, 6].all() and fine[2, 5] and abs(float(ref[2, 5])) > 1e30 and not fine[0, 0]
    for y in (capi.linear_fp4(x, wq, b.to(DEV)), capi.linear_fp4(xq, wq, b.to(DEV)), capi.linear_fp4(x, wq, b.to(DEV), x_scale=scale)):
        y = y.cpu().double()
        assert_within("y", y[fine], ref[fine], tol[fine])
        assert torch.isinf(y[~fine]).all() and torch.equal(y[~fine] > 0, ref[~fine] > 0)
