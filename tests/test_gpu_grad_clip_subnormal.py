"""Clipping of gradients below fp32's normal range, which the norm and the results hold as they hold others.

Bounds as in the tests of the range: 2^-20 for the norm, a few roundings of 2^-24 and the result's own, which below 2^-126 is
half of the smallest step: 2^-150 of fp32, 2^-134 of bf16."""
import math

import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.test_gpu_grad_clip_range import make

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
STEP = {torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 16, 1e30])
@pytest.mark.parametrize("size,max_norm", [(1e-34, 1e9), (1e-37, 1e9), (2e-39, 1e9), (1e-42, 1e9), (1e-34, 1e-33), (1e-36, 1e-38),
                                           (2e-39, 5e-39)])
def test_tiny_gradients(size, max_norm, scale, in_place):
    sizes = (5003, 77, 2049, 8, 1)
    grads = [make(1.0, sizes)[i] for i in range(len(sizes))]
    g = torch.Generator().manual_seed(2)
    grads = [((torch.rand(n, generator=g).double() * 1.9 - 0.95) * size).to(t.dtype).to(DEV) for n, t in zip(sizes, grads)]
    host = [t.cpu().double() for t in grads]
    norm = scale * math.sqrt(sum(float((h * 2.0 ** 130).square().sum()) for h in host)) * 2.0 ** -130
    clip = capi.GradClip(grads, out=None if in_place else [torch.empty_like(t) for t in grads])
    got = clip(max_norm, scale=scale, eps=0.0).cpu().double()
    assert norm > 0.0 and abs(float(got) - norm) <= 2.0 ** -20 * norm + 2.0 ** -149
    factor = scale * min(1.0, max_norm / norm)
    for h, o in zip(host, clip.out):
        want = h * factor
        tol = (2.0 ** -20 + 6 * 2.0 ** -24 + HALF[o.dtype] * 1.01) * want.abs() + STEP[o.dtype]
        assert ((o.cpu().double() - want).abs() <= tol).all()


def test_zero_factor_and_zeros():
    z = [torch.zeros(1000, device=DEV), torch.zeros(33, dtype=torch.bfloat16, device=DEV)]
    assert float(capi.GradClip(z)(1.0)) == 0.0 and all((t == 0).all() for t in z)
    t = [torch.full((1000,), 1e-40, device=DEV)]
    capi.GradClip(t)(0.0)
    assert (t[0] == 0).all()
