"""Clipping by the norm over many gradients on the GPU against fp64: sizes from none to millions at
every alignment, both dtypes together, in place and not, tables of more than a thousand tensors, values
whose squares overflow or vanish, NaN and infinities, streams, replays and the refusals.

Bounds: the squares are summed in fp32 over at most 32 values (32 2^-24 relative, all terms of one
sign) and in 64 bits beyond; the norm is rounded once, the factor is two fp32 operations and a
product, and each result one product and its rounding: 2^-20 covers the norm (64 roundings, halved by
the square root), the factor 2^-20 + 4 2^-24, a result that and its own half step. (Beyond 64 bytes the squares are added in
two fp32 parts, of 48 bits together, and in 64 bits where fp32 does not hold them: the bounds cover either.)"""
import pytest
import torch

from swin_window_attention_gb300 import capi

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def make(sizes, seed=0, std=1e-3, offsets=(0,), dtypes=(torch.float32, torch.bfloat16)):
    """Tensors cut from one buffer a dtype, some elements apart."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = (torch.randn(n + 16, generator=g) * std).to(dtypes[i % len(dtypes)]).to(DEV)
        o = offsets[i % len(offsets)]
        out.append(t[o:o + n])
    return out


def check(grads, max_norm, scale=1.0, out=None, eps=1e-6):
    host = [g.detach().double().cpu() for g in grads]
    norm = scale * sum(float(h.square().sum()) for h in host) ** 0.5
    clip = capi.GradClip(grads, out=out)
    got = clip(max_norm, scale=scale, eps=eps)
    torch.cuda.synchronize()
    assert abs(float(got) - norm) <= 2.0 ** -20 * norm + 1e-44
    factor = scale * min(1.0, max_norm / (norm + eps))
    for h, o in zip(host, clip.out):
        want = h * factor
        tol = (2.0 ** -20 + 4 * 2.0 ** -24 + HALF[o.dtype] * 1.01) * want.abs() + 1e-37
        assert (((o.double().cpu() - want).abs() <= tol).all()), (o.dtype, o.shape)
    return got


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 63, 2047, 2048, 2049, 100001, 3000000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_tensor_every_alignment(n, dtype):
    for off in (range(8) if n < 10 ** 5 else (0, 3)):
        grads = make([n], n, offsets=(off,), dtypes=(dtype,))
        check(grads, 1e-3, out=[torch.empty(n, dtype=dtype, device=DEV)])  # out of another alignment
        check(grads, 1e-3)
        check(grads, 1e9)


@pytest.mark.parametrize("count", [2, 63, 64, 65, 300, 1024, 1025, 2500])
def test_many_tensors(count):
    g = torch.Generator().manual_seed(count)
    sizes = [int(s) for s in torch.randint(0, 5000, (count,), generator=g)]
    sizes[0] = 0
    sizes[1] = 40000
    grads = make(sizes, count, offsets=(0, 1, 5, 2, 7, 3))
    out = [torch.empty_like(t) for t in grads]
    check(grads, 0.01, out=out)
    check(grads, 0.01, scale=0.125)


def test_in_place_leaves_what_is_short_enough():
    grads = make([1000, 77])
    before = [g.clone() for g in grads]
    check(grads, 1e3)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


def test_surroundings_stay():
    for dtype in (torch.float32, torch.bfloat16):
        for off in range(9):
            room = torch.full((5000,), 3.0, dtype=dtype, device=DEV)
            g = room[off:off + 4011]
            capi.GradClip([g])(1.0)
            torch.cuda.synchronize()
            assert (room[:off] == 3).all() and (room[off + 4011:] == 3).all() and (g != 3).all()


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-10, 1e10, 1e18, 1e25, 1e36])
def test_squares_out_of_range(size):
    """Squares below and above what fp32 holds."""
    g = torch.randn(10007, generator=torch.Generator().manual_seed(1)) * size
    check([g.to(DEV), g[:100].bfloat16().to(DEV)], size, eps=0.0)
    mixed = torch.cat([g[:5000], g[5000:] * 1e-6])
    check([mixed.to(DEV)], size, eps=0.0)


def test_zeros_and_no_elements():
    z = torch.zeros(1000, device=DEV)
    assert float(check([z], 1.0)) == 0.0
    e = torch.empty(0, device=DEV)
    n = torch.full((1,), 9.0, device=DEV)
    assert float(capi.GradClip([e, e])(1.0, norm=n)) == 0.0


def test_nan_and_infinity():
    a, b = torch.ones(5000, device=DEV), torch.ones(300, dtype=torch.bfloat16, device=DEV)
    a[17] = float("nan")
    out = [torch.empty_like(a), torch.empty_like(b)]
    n = capi.GradClip([a, b], out=out)(1.0)
    assert torch.isnan(n).all() and all(torch.isnan(o).all() for o in out)
    a[17], b[5] = 1.0, float("-inf")
    n = capi.GradClip([a, b], out=out)(1.0)
    assert torch.isinf(n).all() and (out[0] == 0).all()
    assert torch.isnan(out[1][5]) and (out[1][:5] == 0).all() and (out[1][6:] == 0).all()


def test_other_stream_replay_and_same_bits():
    grads = make([100000, 7, 33333, 4096], 3)
    out = [torch.empty_like(g) for g in grads]
    clip = capi.GradClip(grads, out=out)
    n = clip(0.01)
    first = [o.clone() for o in out]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    n2 = clip(0.01, stream=s, workspace=torch.empty_like(clip.workspace))
    s.synchronize()
    assert torch.equal(n, n2) and all(torch.equal(a, b) for a, b in zip(first, out))
    norm = torch.empty(1, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clip(0.01, norm=norm)
    for g in grads:
        g.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    # twice the gradients: twice the norm, and after clipping the same but for the roundings of eps
    assert torch.equal(norm, 2.0 * n)
    assert all(torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=0.0) for a, b in zip(first, out))


def test_plans_are_dropped_while_another_stream_reads_them():
    """A plan's list outlives its calls on other streams: plans made, called and dropped, while new tensors take their
    memory."""
    s = torch.cuda.Stream()
    grads = make([3000000], 9)
    want = float(grads[0].double().square().sum()) ** 0.5
    torch.cuda.synchronize()
    norms = []
    for _ in range(50):
        clip = capi.GradClip(grads, out=[torch.empty_like(grads[0])])
        norms.append(clip(1.0, stream=s))
        n = clip._room.numel()
        del clip
        torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert all(abs(float(n) - want) < 1e-5 * want for n in norms)


def test_refusals():
    a, b = torch.ones(100, device=DEV), torch.ones(50, device=DEV)
    with pytest.raises(ValueError):
        capi.GradClip([])
    with pytest.raises(ValueError):
        capi.GradClip([a.half()])
    with pytest.raises(ValueError):
        capi.GradClip([a[::2]])
    with pytest.raises(ValueError):
        capi.GradClip([a], out=[b])
    with pytest.raises(ValueError):
        capi.GradClip([a], out=[a.clone(), b])
    for grads, out in (([a, a], None), ([a, a[:10]], None), ([a[:50], a[50:]], [a[25:75], b]), ([a[:50], b], [b, b])):
        with pytest.raises(capi.SwinWAttnError) as e:
            capi.GradClip(grads, out=out)
        assert e.value.status == capi.ERR_INVALID_ARG
    # the same gradient read twice is two gradients
    twice = capi.GradClip([a, a], out=[torch.empty_like(a), torch.empty_like(a)])(1.0)
    assert abs(float(twice) - 200.0 ** 0.5) < 1e-5
    clip = capi.GradClip([a, b])
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0, scale=0.0), dict(max_norm=1.0, eps=-1.0),
               dict(max_norm=float("inf"))):
        with pytest.raises(capi.SwinWAttnError) as e:
            clip(**kw)
        assert e.value.status == capi.ERR_INVALID_ARG
    with pytest.raises(capi.SwinWAttnError):
        clip(1.0, norm=a[3:4])
    with pytest.raises(capi.SwinWAttnError):  # the norm in the plan's own list
        clip(1.0, norm=clip._room[:4].view(torch.float32))
    with pytest.raises(capi.SwinWAttnError):
        clip(1.0, workspace=clip.workspace[:256])
    assert (a == 1).all() and (b == 1).all()
    h = clip.handle
    clip.close()
    assert capi.swin_wattn_clip_destroy(h) == capi.ERR_BAD_PLAN
    with pytest.raises(capi.SwinWAttnError) as e:
        clip(1.0)
    assert e.value.status == capi.ERR_BAD_PLAN
