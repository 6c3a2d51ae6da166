"""NVFP4 with a scale of the tensor that is given: finite blocks saturate however far they lie above it, over the whole
range of given scales, quantised by themselves and inside the product."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.fp4_util import E2M1, E4M3, codes_of, quantize64, scale_bytes_of
from tests.linear_util import assert_within
from tests.test_gpu_fp4 import check_quantized, linear64

pytestmark = pytest.mark.gpu
DEV = "cuda"
HUGE = 3.3e38  # finite in bf16 and in fp32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _rand(seed, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def _spread(ts, dtype):
    """Blocks within the scale's reach, and blocks with values from just beyond it up to the largest finite ones, alone in
    their block and in all of it; one block with an infinity, one with a NaN."""
    x = _rand(1, 40, 128, std=100.0, dtype=torch.float32).double() * ts
    tops = [6.0 * ts * f for f in (447.0, 449.0, 464.0, 465.0, 511.0, 513.0, 2.0 ** 12, 2.0 ** 40)]
    tops += [2.0 ** e for e in range(-60, 128, 11)] + [1.7e9, 3.7e36, HUGE]
    for i, v in enumerate(v for v in tops if v <= HUGE):
        x[i % 38, 16 * (i % 8)] = v if i % 2 else -v
        x[(i + 5) % 38, 16 * ((i + 3) % 8):16 * ((i + 3) % 8) + 16] = -v if i % 3 else v
    x[38, 20], x[39, 100] = float("inf"), float("nan")
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e", [-100, -70, -30, -9, 0, 40, 100])
def test_finite_blocks_saturate(e, dtype):
    """A power of two as scale: every quotient's place among the codes is exact in fp32, so codes and scales are the
    definition's to the bit; only the blocks with an infinity or a NaN are NaN."""
    ts = 2.0 ** e
    x = _spread(ts, dtype)
    q = capi.quantize_fp4(x.to(DEV), "nvfp4", scale=torch.full((1,), ts, device=DEV))
    values = check_quantized(x, "nvfp4", q, ts)
    assert torch.isnan(values).sum() == 32
    back = capi.dequantize_fp4(q, torch.float32).double().cpu()
    assert torch.equal(torch.isnan(back), torch.isnan(values)) and torch.equal(back.nan_to_num(0.0), values.nan_to_num(0.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_finite_blocks_saturate_with_a_calibrated_scale(dtype):
    """Any positive scale: its products and quotients are rounded, by some 2^-22 altogether, so codes are the definition's
    wherever the quotient lies further than that from a border between two."""
    scale = torch.full((1,), 4.8871 / 2688, device=DEV)
    ts = float(scale)
    x = _spread(ts, dtype)
    q = capi.quantize_fp4(x.to(DEV), "nvfp4", scale=scale)
    code, byte, values = quantize64(x, "nvfp4", ts)
    got, clean = scale_bytes_of(q)
    assert clean and torch.equal(got == 0x7F, byte == 0x7F)
    ratio = x.double().reshape(40, 8, 16).abs().amax(-1) / 6.0 / ts
    border = (E4M3[:-1] + E4M3[1:]) / 2
    clear = ((ratio[..., None] / border - 1.0).abs() > 2.0 ** -20).all(-1) & (byte != 0x7F)
    assert torch.equal(got[clear], byte[clear]) and clear.sum() > 300
    step = (E4M3[got.clamp_max(126)] * ts).repeat_interleave(16, -1)
    quotient = x.double().abs() / torch.where(step > 0, step, torch.ones_like(step))
    middle = (E2M1[:-1] + E2M1[1:]) / 2
    sure = clear.repeat_interleave(16, -1) & ((quotient[..., None] / middle - 1.0).abs() > 2.0 ** -20).all(-1)
    assert torch.equal((codes_of(q) & 7)[sure], code[sure]) and sure.sum() > 0.9 * clear.sum() * 16
    back = capi.dequantize_fp4(q, torch.float32).cpu()
    assert torch.equal(torch.isnan(back), torch.isnan(values))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 33, 64, 200])
def test_products_of_such_blocks(T, dtype):
    """Quantised inside the product (few tokens) and before it: no token's result is NaN."""
    K, N, ts = 288, 136, 2.0 ** -9
    x = _rand(T, T, K, dtype=dtype)
    x[0, 35], x[T // 2, 287], x[T - 1, 64:80] = HUGE, -HUGE, HUGE
    wq = capi.quantize_fp4(_rand(2, N, K, std=K ** -0.5).to(DEV), "nvfp4")
    wv = capi.dequantize_fp4(wq, torch.float32).double().cpu()
    scale = torch.full((1,), ts, device=DEV)
    y = capi.linear_fp4(x.to(DEV), wq, x_scale=scale)
    torch.cuda.synchronize()
    assert_within("y", y, *linear64(quantize64(x, "nvfp4", ts)[2], wv, None, "none", None))
    calibrated = torch.full((1,), 4.8871 / 2688, device=DEV)
    assert torch.isfinite(capi.linear_fp4(x.to(DEV), wq, x_scale=calibrated)).all()
