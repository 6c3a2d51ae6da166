"""Weight updates of low rank and of falling singular values on the GPU, as raw gradients and
momenta are, against the Newton-Schulz iteration in fp64: within the bound that the header
states, which does not follow from how the kernels round."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.linear_util import HALF_BF16, NS, orthogonalize64
from tests.orthogonalize_util import BOUND, assert_update, matrix

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _run(g, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = capi.orthogonalize(g.to(DEV), status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return out.cpu().double()


KINDS = ["flat", "log", "half", "power1", "power1.5", "power2", "rank1", "rank16", "rank49"]


# one CTA; its largest; a cluster; its largest; separate products; with the Gram product in parts
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(96, 200), (96, 384), (385, 128), (70, 1500), (2048, 128), (200, 264), (530, 384),
                                 (150, 3000), (100, 2049)])
def test_against_fp64(kind, m, n):
    g = matrix(kind, m, n, seed=m + n)
    assert_update(_run(g), g, orthogonalize64(g, 5), 5)
    t = g.T.contiguous()
    assert_update(_run(t), t, orthogonalize64(t, 5), 5)


@pytest.mark.parametrize("kind,m,n", [("rank49", 512, 2048), ("rank16", 1000, 1536), ("half", 384, 1152)])
def test_larger_ones(kind, m, n):
    g = matrix(kind, m, n)
    assert_update(_run(g), g, orthogonalize64(g, 5), 5)


@pytest.mark.parametrize("m,n", [(96, 384), (1024, 80), (260, 300)])
def test_each_matrix_of_a_stack(m, n):
    kinds = ("rank1", "flat", "power1.5", "half", "rank49")
    g = torch.stack([matrix(k, m, n, seed=i) for i, k in enumerate(kinds)])
    out = _run(g)
    for o, x in zip(out, g):
        assert_update(o, x, orthogonalize64(x, 5), 5)


@pytest.mark.parametrize("m,n", [(96, 384), (200, 512)])
@pytest.mark.parametrize("tokens", [1, 49, 100])
def test_gradient_of_a_few_tokens(tokens, m, n):
    """A gradient as linear_bwd_weight leaves it, of rank `tokens` at most, and its update."""
    gen = torch.Generator().manual_seed(tokens)
    dy = (1e-3 * torch.randn(tokens, m, generator=gen)).bfloat16().to(DEV)
    x = torch.randn(tokens, n, generator=gen).bfloat16().to(DEV)
    dw, _ = capi.linear_bwd_weight(dy, x)
    g = dw.cpu()
    assert_update(_run(g), g, orthogonalize64(g, 5), 5)


@pytest.mark.parametrize("m,n", [(96, 300), (160, 200)])
def test_empty_directions_stay_empty(m, n):
    """A gradient of rank r keeps its row space: what of the result lies outside is at most its
    roundings, 2^-8 of the entries and the noise of the products that make it."""
    g = matrix("rank5", m, n)
    out = _run(g)
    v = torch.linalg.svd(g.double(), full_matrices=False)[2][:5]
    outside = out - (out @ v.T) @ v
    assert float(outside.norm()) <= 2.0 ** -8 * float(out.norm()) * 1.01


@pytest.mark.parametrize("kind", ["rank49", "half", "power2"])
def test_seven_steps(kind):
    """Two more steps, in which noise that the first left has grown by 3.44 each: twice the bound."""
    for m, n in ((96, 384), (200, 264)):
        g = matrix(kind, m, n)
        assert_update(_run(g, steps=7), g, orthogonalize64(g, 7), 7, bound=4e-3)


@pytest.mark.parametrize("m,n", [(2, 9), (3, 100), (5, 8), (8, 64), (16, 16), (40, 16), (32, 300), (3, 9000)])
def test_few_rows(m, n):
    """Few rows average their roundings less: the header's bounds for them."""
    for kind in ("rank1", "flat", "power1", "half"):
        g = matrix(kind, m, n, seed=m)
        assert_update(_run(g), g, orthogonalize64(g, 5), 5, bound=6e-3 if min(m, n) < 32 else 4e-3,
                      model=False)


def test_largest_matrix():
    """One step of the largest sides, on sampled rows: with y = x_r X^T, row r of A, the result's row is
    a x_r + b y X + c ((y X) X^T) X."""
    a, b, c = NS
    n = 16384
    gen = torch.Generator(device=DEV).manual_seed(1)
    g = torch.randn(n, n, generator=gen, device=DEV)
    out = capi.orthogonalize(g, steps=1, status=(st := torch.zeros(1, dtype=torch.int32, device=DEV)))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    rows = torch.tensor([0, 1, 255, 256, 8191, 12345, 16383], device=DEV)
    x = g.double()
    x /= x.norm()
    xr = x[rows]
    z = (xr @ x.T) @ x
    exact = a * xr + b * z + c * ((z @ x.T) @ x)
    err = (out[rows].double() - exact).norm(dim=1) / exact.norm(dim=1)
    assert float(err.max()) <= BOUND + HALF_BF16 * (1.0 + BOUND)
