"""Clipping where the factor, or the norm itself, lies outside of what fp32 holds: finite gradients come out with the norm
that was asked for.

Bounds: the squares are summed in fp32 over the values of 64 bytes (at most 32 of them, roundings of 2^-24 each) and in two
fp32 parts or in 64 bits beyond, whose errors are below 2^-40: the sum is off by 2^-19 at most, its root by 2^-20. The factor
is rounded a few times, a result once or twice in fp32 and once to its type. What is below 2^-126 may be flushed to zero."""
import math

import pytest
import torch

from swin_window_attention_gb300 import capi

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32_MAX = 3.4028235e38


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def check(grads, max_norm, scale=1.0, eps=1e-6, in_place=True):
    host = [g.double().cpu() for g in grads]
    root = math.sqrt(sum(float((h * 2.0 ** -100).square().sum()) for h in host)) * 2.0 ** 100
    norm = scale * root
    clip = capi.GradClip(grads, out=None if in_place else [torch.empty_like(g) for g in grads])
    got = float(clip(max_norm, scale=scale, eps=eps))
    if norm < 0.999 * F32_MAX:
        assert abs(got - norm) <= 2.0 ** -20 * norm + 2.0 ** -126
    elif norm > 1.001 * F32_MAX:
        assert got == float("inf")
    factor = scale * min(1.0, max_norm / (norm + eps))
    for h, o in zip(host, clip.out):
        want = h * factor
        tol = (2.0 ** -20 + 6 * 2.0 ** -24 + HALF[o.dtype] * 1.01) * want.abs() + 2.0 ** -126
        o = o.double().cpu()
        assert torch.isfinite(o).all() and ((o - want).abs() <= tol).all()
        assert float(o.abs().max()) > 0.0 or float(want.abs().max()) < 2.0 ** -120


def make(size, sizes=(5003, 77, 2049)):
    g = torch.Generator().manual_seed(1)
    out = []
    for i, n in enumerate(sizes):
        t = (torch.rand(n, generator=g) * 1.9 - 0.95) * size
        out.append(t.to(torch.bfloat16 if i % 2 else torch.float32).to(DEV))
    return out


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("size,max_norm", [(1e36, 0.25), (1e36, 1e-3), (1e38, 1e-30), (3e37, 1.0), (1e20, 1e-19), (1e30, 1e-20)])
def test_factor_below_fp32(size, max_norm, in_place):
    check(make(size), max_norm, in_place=in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("max_norm", [1.0, 1e-6, 1e30, 3e38])
def test_norm_beyond_fp32(max_norm, in_place):
    check(make(3e38), max_norm, in_place=in_place)


@pytest.mark.parametrize("size,scale", [(1e10, 1e35), (1e3, 1e38), (1.0, 2.0 ** -100), (1e36, 2.0 ** -16), (1e-30, 2.0 ** -90)])
def test_scales(size, scale):
    """The norm is scale times the root: both may be ordinary and their product not."""
    check(make(size), 2.0 if scale > 1.0 else 1e-30, scale=scale, eps=0.0, in_place=False)


def test_infinities_and_zeros_as_before():
    a = torch.full((300,), 1e38, device=DEV)
    a[7] = float("inf")
    n = capi.GradClip([a])(1.0)
    assert torch.isinf(n).all() and torch.isnan(a[7]) and (a[:7] == 0).all() and (a[8:] == 0).all()
    b = torch.full((300,), 1e38, device=DEV)
    capi.GradClip([b])(0.0)
    assert (b == 0).all()


def test_replayed():
    """Ordinary values and such ones through the same captured call."""
    g = make(1.0)
    clip = capi.GradClip(g)
    norm = torch.empty(1, device=DEV)
    clip(0.5, norm=norm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clip(0.5, norm=norm)
    for size in (1e37, 1.0, 3e38):
        src = make(size)
        want = make(size)
        capi.GradClip(want)(0.5)
        for t, s in zip(g, src):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(g, want))
        total = math.sqrt(sum(float(t.double().square().sum()) for t in g))
        assert abs(total - 0.5) < 0.5 * 2.0 ** -8
