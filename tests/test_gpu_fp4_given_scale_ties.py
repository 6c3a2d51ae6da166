"""NVFP4 with the smallest and the largest scales that may be given: borders between two roundings, whose quotients' remainders
lie below fp32's normal range there."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.fp4_util import E2M1, E4M3
from tests.test_gpu_fp4 import check_quantized

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _borders(ts, dtype):
    """A block for each scale of E4M3 but zero and each border between two codes: the border, the numbers next to it, and six
    times the scale; and blocks whose largest value lies on a border between two scales, and next to it."""
    steps = E4M3[1:] * ts
    t = (E2M1[:-1] + E2M1[1:]) / 2
    blocks = torch.zeros(len(steps), len(t), 16, dtype=torch.float64)
    blocks[..., 0] = steps[:, None] * t
    blocks[..., 15] = 6.0 * steps[:, None]
    b = blocks.to(dtype)
    up = torch.tensor(float("inf"), dtype=dtype)
    b[..., 1], b[..., 2] = torch.nextafter(b[..., 0], up), torch.nextafter(b[..., 0], -up)
    b[..., 3:6] = -b[..., 0:3]
    top = (6.0 * (E4M3[:-1] + E4M3[1:]) / 2 * ts).to(dtype)
    tops = torch.stack([top, torch.nextafter(top, up), torch.nextafter(top, -up)], 1).reshape(-1)
    c = tops[:, None] * torch.linspace(-1.0, 1.0, 16).to(dtype)
    c[:, 7] = tops
    x = torch.cat([b.reshape(-1, 16), c])
    return x[:len(x) // 8 * 8].reshape(-1, 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e", [-100, -99, -98, -95, -90, -40, 60, 100])
def test_borders(e, dtype):
    """To the bit: with a power of two as scale every border is a number of few bits, and the definition's quotients are
    exact there."""
    ts = 2.0 ** e
    x = _borders(ts, dtype)
    q = capi.quantize_fp4(x.to(DEV), "nvfp4", scale=torch.full((1,), ts, device=DEV))
    values = check_quantized(x, "nvfp4", q, ts)
    assert torch.equal(capi.dequantize_fp4(q, torch.float32).double().cpu(), values)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e", [-100, -99])
def test_random_values(e, dtype):
    g = torch.Generator().manual_seed(3)
    for std in (0.05, 1.0, 300.0):
        x = (torch.randn(400, 1280, generator=g).double() * std * 2.0 ** e).to(dtype)
        q = capi.quantize_fp4(x.to(DEV), "nvfp4", scale=torch.full((1,), 2.0 ** e, device=DEV))
        check_quantized(x, "nvfp4", q, 2.0 ** e)
