"""What the activations give at and near -inf, +inf and zero, in both forms of the products."""
import pytest
import torch

from swin_window_attention_gb300 import capi

pytestmark = pytest.mark.gpu
DEV = "cuda"
Z = [float("-inf"), -1e30, -200.0, -90.0, -15.0, -14.0, 0.0, 15.0, 200.0, 1e30, float("inf"), float("nan")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


@pytest.mark.parametrize("T", [3, 2000])  # clusters; tiles
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_far_values(act, T):
    """z through the bias: 0 where the exact value rounds to 0 in fp32 (z below -14 for
    the GELUs, below -100 for SiLU), z itself far on the right, NaN kept."""
    n = 16
    b = torch.zeros(n, device=DEV)
    b[:len(Z)] = torch.tensor(Z)
    x, w = torch.zeros(T, 8, dtype=torch.bfloat16, device=DEV), torch.zeros(n, 8, dtype=torch.bfloat16, device=DEV)
    y = capi.linear(x, w, b, act=act).float().cpu()
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(y, nan=7.0), torch.nan_to_num(y[:1], nan=7.0).expand_as(y))
    far = [i for i, z in enumerate(Z) if z <= (-200.0 if act == "silu" else -14.0)]
    assert all(float(y[0, i]) == 0.0 for i in far), y[0]
    for i, z in enumerate(Z):
        if z >= 15.0:
            assert float(y[0, i]) == float(torch.tensor(z).bfloat16())
    assert float(y[0, Z.index(0.0)]) == 0.0 and torch.isnan(y[0, len(Z) - 1])
