"""Orthogonalised weight updates on the GPU against the Newton-Schulz iteration in fp64: the
error may be a quarter above that of the same iteration in fp64 with the held matrices
rounded to fp16 and the result to bf16 (what the kernels' fp32 accumulation adds to those
roundings is a thousandth of them; a quarter leaves room for roundings that fall the other
way), and the properties of the result that do not need the iteration."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.linear_util import orthogonalize64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _g(seed, *shape, dtype=torch.float32, strong=0.5):
    gen = torch.Generator().manual_seed(seed)
    n, r, c = shape
    k = min(4, r, c)
    low = torch.randn(n, r, k, generator=gen) @ torch.randn(n, k, c, generator=gen)
    return ((strong * low + torch.randn(n, r, c, generator=gen)) * 1e-3).to(dtype)


def _run(g, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = capi.orthogonalize(g.to(DEV), status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert out.dtype == torch.bfloat16 and out.shape == g.shape
    return out.cpu().double()


def _check(out, g, steps=5, scale=1.0):
    for o, m in zip(out, g):
        exact = orthogonalize64(m, steps, scale=scale)
        held = orthogonalize64(m, steps, scale=scale, half=True)
        err, allow = float((o - exact).norm()), float((held - exact).norm())
        assert err <= 1.25 * allow + 1e-4 * float(exact.norm()), (err, allow, float(exact.norm()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,r,c", [(1, 96, 384), (1, 384, 96), (3, 64, 64), (2, 200, 136), (2, 136, 200), (5, 33, 77),
                                   (4, 77, 33), (1, 129, 513), (1, 512, 300), (7, 24, 1000), (2, 700, 40),
                                   (40, 130, 264), (1, 1024, 640), (2, 128, 2049), (1, 4096, 128),
                                   (1, 100, 4000), (3, 1500, 97), (20, 128, 512), (1, 128, 4104), (2, 129, 96),
                                   (16, 50, 700), (30, 640, 33), (1, 20, 513), (80, 16, 600)])
def test_against_fp64(n, r, c, dtype):
    g = _g(n + r + c, n, r, c, dtype=dtype)
    _check(_run(g), g)


@pytest.mark.parametrize("n,r,c", [(40, 333, 340), (40, 390, 384), (30, 264, 530), (4, 777, 800), (4, 810, 777),
                                   (2, 1100, 1101)])
def test_only_half_of_the_symmetric_products(n, r, c):
    """Stacks large enough that only the tiles on and below the diagonal of A and B are computed."""
    g = _g(n + r, n, r, c)
    out = _run(g)
    pick = [0, n // 2, n - 1]
    _check(out[pick], g[pick])
    # the same matrices one at a time, where all tiles may be computed (each within 2^-9 of the exact)
    one = torch.cat([_run(g[k:k + 1]) for k in pick])
    assert float((one - out[pick]).norm() / one.norm()) < 2.0 ** -8


@pytest.mark.parametrize("n,r,c", [(2, 70, 5497), (2, 5496, 71), (1, 135, 3341), (1, 300, 6000), (3, 2500, 131),
                                   (1, 16384, 40), (1, 1, 16384), (1, 4097, 1)])
def test_gram_product_in_parts(n, r, c):
    """Few tiles of a long product: its parts are summed in a launch of their own."""
    g = _g(n + r, n, r, c)
    _check(_run(g), g)


@pytest.mark.parametrize("r,c,steps", [(540, 126, 6), (96, 384, 5), (62, 588, 6), (300, 310, 6), (1400, 100, 7),
                                       (100, 500, 12), (520, 140, 6), (1, 40, 5), (24, 64, 1), (24, 64, 20)])
def test_error_beside_the_rounding_of_the_result(r, c, steps):
    """Against the iteration in fp64 with the same matrices rounded (the quarter as above), and, up
    to seven steps, no further off than half as far again as rounding the exact result to bf16."""
    g = _g(3 * r + c, 2, r, c)
    out = _run(g, steps=steps)
    for o, m in zip(out, g):
        exact, held = orthogonalize64(m, steps), orthogonalize64(m, steps, half=True)
        err, size = float((o - exact).norm()), float(exact.norm())
        assert err <= 1.25 * float((held - exact).norm()) + 1e-4 * size
        if steps <= 7:
            assert err <= 1.5 * float((exact.to(torch.bfloat16).double() - exact).norm()) + 1e-4 * size


@pytest.mark.parametrize("steps,scale", [(1, 1.0), (2, 0.25), (3, -2.0), (8, 1.7)])
def test_steps_and_scale(steps, scale):
    g = _g(steps, 2, 96, 160)
    _check(_run(g, steps=steps, scale=scale), g, steps, scale)


@pytest.mark.parametrize("r,c", [(40, 96), (140, 150)])
def test_smallest_and_largest_scales(r, c):
    g = _g(r, 1, r, c)
    for scale in (2.0 ** -100, -(2.0 ** 100), 0.0):
        _check(_run(g, scale=scale), g, scale=scale)


@pytest.mark.parametrize("r,c", [(1, 1), (1, 7), (9, 1), (1, 1000), (8, 8), (2, 3)])
def test_smallest_sizes(r, c):
    g = _g(r + c, 3, r, c)
    _check(_run(g), g)


def test_two_dimensions_and_singular_values():
    g = _g(5, 1, 192, 768)[0]
    o = _run(g)
    s = torch.linalg.svdvals(o)
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25
    # U and V are kept: O G^T is near symmetric and positive
    p = o @ g.double().T
    assert float((p - p.T).norm() / p.norm()) < 2e-2 and float(torch.linalg.eigvalsh(p + p.T).min()) > 0


def test_scale_of_the_input_does_not_matter():
    """eps is 4e-7 of the unscaled norm: below the roundings, so the result for G holds for f G."""
    g = _g(6, 1, 100, 136)
    for f in (2.0 ** 40, 2.0 ** 80, 2.0 ** 100):  # squares that overflow fp32 beyond 2^64
        _check(_run(g * f), g)


@pytest.mark.parametrize("r,c", [(100, 136), (1200, 30), (140, 200)])
def test_small_values(r, c):
    """Values whose squares are no fp32 numbers, with an eps as much smaller, and one scale at
    which values lie on both sides of the bound between two ranges of the norm's sum. The exact
    result is that of G and eps times the same power of two, here in 64 bits."""
    for dtype in (torch.float32, torch.bfloat16):
        g = _g(r, 2, r, c, dtype=dtype)
        for f in (2.0 ** -38, 2.0 ** -60, 2.0 ** -80, 2.0 ** -100):
            _check(_run(g * f, eps=1e-7 * f), g)
    # |G| far below eps: X small from the start, where fp16 holds fewer bits
    g = _g(r, 2, r, c) * 2.0 ** -40
    _check(_run(g), g)


@pytest.mark.parametrize("r,c", [(100, 136), (1200, 30), (140, 200)])
def test_one_value_at_the_ends_of_the_range(r, c):
    """A matrix of one entry keeps to the iteration on that number. Per step the roundings of A,
    of the polynomial and of the result to fp16 (2^-11 of each) change it by less than 4 x 2^-11,
    as |x| <= 1.2 and x A |b + 2 c A| < 1.7; the steps after it multiply that by their slopes."""
    at = [(2.0 ** -126, 3, 5), (2.0 ** 127, 2, 1), (-(2.0 ** -64), 7, 7)]
    g = torch.zeros(3, r, c)
    for m, (v, i, j) in enumerate(at):
        g[m, i, j] = v
    out = _run(g, eps=2.0 ** -126)
    for m, (v, i, j) in enumerate(at):
        s, err = abs(v) / (abs(v) + 2.0 ** -126), 0.0
        for _ in range(5):
            slope = 3.4445 - 3 * 4.7750 * s ** 2 + 5 * 2.0315 * s ** 4
            s, err = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5, abs(slope) * err + 4 * 2.0 ** -11
        got = float(out[m, i, j]) * (1 if v > 0 else -1)
        assert abs(got - s) <= err + 2.0 ** -8 * (s + err), (m, got, s, err)
        out[m, i, j] = 0.0
    assert torch.all(out == 0)
    assert torch.all(_run(torch.zeros(1, r, c), eps=2.0 ** -126) == 0)


def test_zero_and_non_finite_matrices_leave_the_others_alone():
    g = _g(7, 4, 72, 96)
    ref = _run(g)
    g[1] = 0.0
    g[2, 3, 5] = float("nan")
    out = _run(g)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[3], ref[3])
    assert torch.all(out[1] == 0) and torch.isnan(out[2]).all()
    g[2, 3, 5] = float("inf")
    assert torch.isnan(_run(g)[2]).any()


def test_unaligned_rows_write_only_the_result():
    n, r, c = 2, 50, 37
    g = _g(8, n, r, c)
    buf = torch.full((n * r * c + 41,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[21:21 + n * r * c].view(n, r, c)
    capi.orthogonalize(g.to(DEV), out=out)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().double(), _run(g))
    assert torch.all(buf[:21] == 7.0) and torch.all(buf[21 + n * r * c:] == 7.0)
    # an aligned shape at an address that is not
    g = _g(9, 1, 40, 64)
    out = buf[1:1 + 40 * 64].view(1, 40, 64)
    capi.orthogonalize(g.to(DEV), out=out)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().double(), _run(g))


def test_streams_graph_and_empty_stack():
    g = [_g(s, 3, 96, 128).to(DEV) for s in (1, 2)]
    want = [capi.orthogonalize(a) for a in g]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [capi.orthogonalize(a, stream=s) for a, s in zip(g, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = g[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = capi.orthogonalize(x)
    x.copy_(g[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1])
    assert capi.orthogonalize(torch.empty(0, 8, 8, device=DEV)).shape == (0, 8, 8)


def test_error_paths():
    g = torch.zeros(2, 16, 24, device=DEV)
    out = torch.full((2, 16, 24), 3.0, dtype=torch.bfloat16, device=DEV)
    need = capi.swin_wattn_orthogonalize_workspace_bytes(2, 16, 24)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    s = torch.cuda.current_stream().cuda_stream

    def f(gp=g.data_ptr(), op=out.data_ptr(), n=2, r=16, c=24, dt=capi.FP32, steps=5, eps=1e-7, scale=1.0,
          wp=ws.data_ptr(), nb=need):
        return capi.swin_wattn_orthogonalize(gp, op, n, r, c, dt, steps, eps, scale, wp, nb, None, s)

    bad = capi.ERR_INVALID_ARG
    assert f(n=0) == capi.OK and f(n=-1) == bad and f(n=65536) == capi.ERR_UNSUPPORTED
    assert f(r=0) == capi.ERR_UNSUPPORTED and f(c=16385) == capi.ERR_UNSUPPORTED
    assert f(steps=0) == bad and f(steps=21) == bad and f(eps=0.0) == bad and f(eps=float("nan")) == bad
    assert f(scale=float("inf")) == bad and f(dt=4) == bad and f(nb=need - 1) == bad
    assert f(gp=None) == bad and f(op=g.data_ptr()) == bad and f(op=ws.data_ptr()) == bad
    assert f(gp=g.data_ptr() + 2) == capi.ERR_MISALIGNED and f(wp=ws.data_ptr() + 8) == capi.ERR_MISALIGNED
    torch.cuda.synchronize()
    assert torch.all(out == 3.0)
    with pytest.raises(ValueError):
        capi.orthogonalize(g.half())
    with pytest.raises(ValueError):
        capi.orthogonalize(g.transpose(1, 2))
    with pytest.raises(ValueError):
        capi.orthogonalize(g, out=torch.empty(2, 16, 24, device=DEV))
