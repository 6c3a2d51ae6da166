"""linear_fp4 on fp32 activations, and on activations quantised inside the product with a given scale: exact on operands that
4 bits hold, and against fp64 elsewhere."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.fp4_util import exact_operand, quantize64
from tests.linear_util import assert_within
from tests.test_gpu_fp4 import linear64

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _rand(seed, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


# few tokens (one turn of a block's threads over a chunk, several, with idle threads), many; K that ends inside a step, inside
# a chunk and behind one
SHAPES = [(1, 32, 8), (1, 1536, 264), (2, 96, 40), (17, 160, 264), (31, 2080, 128), (32, 256, 72), (33, 288, 136), (49, 1536, 512), (64, 64, 64),
          (64, 544, 2000), (65, 384, 136), (100, 384, 1152), (128, 224, 96), (300, 32, 1000), (1025, 480, 200)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_exact(T, K, N, dtype, fmt):
    """Every sum is a multiple of 1/4 below 2^22: the results are known to the bit."""
    x, w = exact_operand(T, T, K, fmt).to(dtype), exact_operand(N + 1, N, K, fmt)
    b = torch.randint(-9, 10, (N,), generator=torch.Generator().manual_seed(3)).float()
    r = torch.randint(-50, 51, (T, N), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    wq = capi.quantize_fp4(w.to(DEV), fmt)
    z = x.double() @ w.double().T
    want, more = z.to(torch.bfloat16), ((z + b.double()).clamp_min(0) + r.double()).to(torch.bfloat16)
    # the blocks' scales, 1, 2 and 4 over the tensor's, are E4M3 numbers for each of these
    scales = [None] + ([torch.full((1,), s, device=DEV) for s in (1.0, 0.25, 2.0 ** 8)] if fmt == "nvfp4" else [])
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    for s in scales:
        y = capi.linear_fp4(x.to(DEV), wq, x_scale=s, status=st)
        y2 = capi.linear_fp4(x.to(DEV), wq, b.to(DEV), act="relu", residual=r.to(DEV), x_scale=s, status=st)
        torch.cuda.synchronize()
        assert int(st) == 0 and torch.equal(y.cpu(), want) and torch.equal(y2.cpu(), more)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,N", [(1, 224, 120), (20, 1536, 96), (50, 384, 1536), (333, 128, 264), (5, 1536, 6144)])
def test_against_fp64(T, K, N, fmt):
    x, w, b, r = _rand(T, T, K), _rand(1, N, K, std=2.0 * K ** -0.5), _rand(2, N), _rand(3, T, N, dtype=torch.bfloat16)
    wq = capi.quantize_fp4(w.to(DEV), fmt)
    wv = capi.dequantize_fp4(wq, torch.float32).double().cpu()
    for ts in ((None, 2.0 ** -9) if fmt == "nvfp4" else (None,)):
        xq = capi.quantize_fp4(x.to(DEV), fmt)
        s = float(xq.tensor_scale) if fmt == "nvfp4" and ts is None else ts
        xv = quantize64(x, fmt, s)[2]
        scale = None if ts is None else torch.full((1,), ts, device=DEV)
        for act in ("none", "gelu"):
            y = capi.linear_fp4(x.to(DEV), wq, b.to(DEV), act=act, residual=r.to(DEV), x_scale=scale)
            torch.cuda.synchronize()
            assert_within("y", y, *linear64(xv, wv, b, act, r))


@pytest.mark.parametrize("T", [5, 60, 200])
def test_non_finite_values_stay_in_their_token(T):
    for fmt in FORMATS:
        x, wq = _rand(1, T, 320), capi.quantize_fp4(_rand(2, 72, 320).to(DEV), fmt)
        scale = torch.full((1,), 2.0 ** -9, device=DEV) if fmt == "nvfp4" else None
        ref = capi.linear_fp4(x.to(DEV), wq, x_scale=scale)
        x[3, 9], x[T - 1, 319] = float("nan"), float("-inf")
        y = capi.linear_fp4(x.to(DEV), wq, x_scale=scale)
        keep = torch.ones(T, dtype=torch.bool)
        keep[3] = keep[T - 1] = False
        assert torch.equal(y.cpu()[keep], ref.cpu()[keep]) and torch.isnan(y[3]).all() and torch.isnan(y[T - 1]).all()
