"""The residual sum with its norms, gate and stochastic depth, and its gradients, on the GPU against
plain fp64 forms: every row shape, both streams, every combination of parts, results in place,
untouched surroundings, rows with NaN, other streams, graph replays and the refusals."""
import itertools

import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.block_norm_util import assert_close, backward64, forward64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


class Case:
    def __init__(self, T, C, stream=torch.bfloat16, kind="layer", block=True, pre=True, post=True, gate=True, samples=0,
                 alpha=1.0, dy=True, bias=True, seed=0, eps=1e-5):
        g = torch.Generator().manual_seed(seed + 1000 * T + C)

        def n(*s, std=1.0, mean=0.0):
            return torch.randn(*s, generator=g) * std + mean

        self.kind, self.alpha, self.eps, self.stream = kind, alpha, eps, stream
        self.x = (n(T, C) + n(C, std=0.5) + 0.3).to(stream)
        self.f = n(T, C, std=0.7).bfloat16() if block else None
        self.pre = (n(C, std=0.2, mean=1.0), n(C, std=0.3) if bias else None) if pre else None
        self.post = (n(C, std=0.2, mean=1.0), n(C, std=0.3) if bias else None) if post and block else None
        self.gate = n(C, std=0.3, mean=0.5) if gate and block else None
        self.keep = torch.where(torch.rand(samples, generator=g) < 0.7, 1.25, 0.0) if samples and block else None
        self.dh = n(T, C, std=1e-2).bfloat16() if pre else None
        self.dy = n(T, C, std=1e-2).to(stream) if dy or not pre else None

    def parts(self, dev=None):
        to = (lambda t: t) if dev is None else (lambda t: None if t is None else t.to(dev))
        pair = lambda p: None if p is None else (to(p[0]), to(p[1]))
        return dict(pre=pair(self.pre), post=pair(self.post), gate=to(self.gate), keep=to(self.keep), alpha=self.alpha,
                    kind=self.kind, eps=self.eps)

    def check_forward(self, **more):
        f = None if self.f is None else self.f.to(DEV)
        y, h = capi.block_norm(self.x.to(DEV), f, **self.parts(DEV), **more)
        torch.cuda.synchronize()
        want_y, want_h = forward64(self.x, self.f, stream=self.stream, **self.parts())
        assert (y is None) == (want_y is None) and (h is None) == (want_h is None)
        if y is not None:
            assert y.dtype == self.stream
            assert_close("y", y, want_y)
        if h is not None:
            assert h.dtype == torch.bfloat16
            assert_close("h", h, want_h)
        return y, h

    def check_backward(self, **more):
        to = lambda t: None if t is None else t.to(DEV)
        dx, df, grads = capi.block_norm_bwd(self.x.to(DEV), to(self.f), dh=to(self.dh), dy=to(self.dy), **self.parts(DEV),
                                            **more)
        torch.cuda.synchronize()
        want = backward64(self.x, self.f, self.dh, self.dy, stream=self.stream, **self.parts())
        assert_close("dx", dx, want.pop("dx"))
        assert (df is None) == (self.f is None)
        if df is not None:
            assert_close("df", df, want.pop("df"))
        assert set(grads) == set(want)
        for k, v in want.items():
            assert_close(k, grads[k], v)
        return dx, df, grads


# every row shape: groups of 4 to 32 threads with two and three chunks, blocks, with and without idle
# chunks; rows that fill a block of threads, one more, and a single one
WIDTHS = [8, 24, 64, 72, 96, 128, 136, 192, 200, 256, 264, 384, 392, 512, 520, 768, 776, 1000, 1536, 2048, 4104, 8192]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("T", [1, 33, 130])
def test_forward_every_width(C, T):
    Case(T, C, samples=1).check_forward()


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("T", [1, 33, 130])
def test_backward_every_width(C, T):
    Case(T, C, samples=1).check_backward()


@pytest.mark.parametrize("T,C", [(3001, 96), (5000, 8), (700, 1536), (400, 8192), (1999, 768)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_many_tokens(T, C, stream):
    c = Case(T, C, stream=stream, samples=T if T == 1999 else 0)
    c.check_forward()
    c.check_backward()


# rows enough for the form that walks rows, in every row shape of its, a few more than fill its blocks evenly
WALKED = [(116741, 8), (120003, 24), (116735, 40), (58403, 64), (58371, 96), (60000, 104), (29185, 128), (30001, 192), (14600, 256),
          (14599, 264), (16000, 384), (10947, 512), (7299, 520), (9121, 768), (5475, 776), (7003, 1024), (5473, 1032), (6001, 1536)]


@pytest.mark.parametrize("T,C", WALKED)
def test_many_rows(T, C):
    for i, block, post, gate, pre, kind in [(0, 1, 1, 1, 1, "layer"), (1, 1, 0, 1, 1, "layer"), (2, 1, 0, 0, 1, "rms"), (3, 0, 0, 0, 1, "layer"),
                                            (4, 1, 1, 0, 0, "rms")]:
        c = Case(T, C, kind=kind, block=block, post=post, gate=gate, pre=pre, samples=T if i < 2 else 0, alpha=1.0 if i else -2.5,
                 bias=i != 2)
        c.x[T // 2, 3], c.x[T - 1, C - 1] = float("nan"), float("-inf")
        x, f = c.x.to(DEV), None if c.f is None else c.f.to(DEV)
        y, h = capi.block_norm(x.clone(), f, **c.parts(DEV))
        want = forward64(x, f, stream=c.stream, **c.parts(DEV))
        fine = torch.ones(T, dtype=torch.bool, device=DEV)
        fine[T // 2] = fine[T - 1] = False
        for name, got, w in (("y", y, want[0]), ("h", h, want[1])):
            assert (got is None) == (w is None)
            if got is not None:
                assert_close(name, got[fine], (w[0][fine].cpu(), w[1][fine].cpu()))
                assert torch.equal(torch.isnan(got), torch.isnan(w[0]))
        if block:  # over x, between guards
            room = torch.zeros(T + 2, C, dtype=torch.bfloat16, device=DEV)
            room[1:-1] = x
            again, h2 = capi.block_norm(room[1:-1], f, y=room[1:-1], **c.parts(DEV))
            assert torch.equal(again.view(torch.int16), y.view(torch.int16))
            assert h is None or torch.equal(h2.view(torch.int16), h.view(torch.int16))
            assert (room[0] == 0).all() and (room[-1] == 0).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("pre,post,gate,samples,bias,dy", list(itertools.product([0, 1], [0, 1], [0, 1], [0, 3], [0, 1], [0, 1])))
def test_every_combination(kind, pre, post, gate, samples, bias, dy):
    for stream in (torch.bfloat16, torch.float32):
        c = Case(21, 200, stream, kind, True, pre, post, gate, samples, 1.0 if bias else -2.5, dy, bias)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_plain_norm(kind, stream):
    for T, C in [(1, 1536), (49, 96), (77, 1000)]:
        for dy in (0, 1):
            c = Case(T, C, stream, kind, block=False, dy=dy)
            c.check_forward()
            c.check_backward()


def test_leading_axes_and_given_results():
    c = Case(24, 96, samples=2)
    x, f = c.x.view(2, 3, 4, 96).to(DEV), c.f.view(2, 3, 4, 96).to(DEV)
    y, h = torch.empty_like(x), torch.empty_like(f)
    a, b = capi.block_norm(x, f, y=y, h=h, **c.parts(DEV))
    assert a is y and b is h
    want_y, want_h = forward64(c.x, c.f, stream=c.stream, **c.parts())
    assert_close("y", y.view(24, 96), want_y)
    assert_close("h", h.view(24, 96), want_h)
    grads = {"gate": torch.full((96,), 2.0, device=DEV), "pre_bias": torch.full((96,), -1.0, device=DEV)}
    _, _, got = capi.block_norm_bwd(x, f, dh=c.dh.view_as(x).to(DEV), dy=c.dy.view_as(x).to(DEV), grads=grads, accumulate=True,
                                    **c.parts(DEV))
    want = backward64(c.x, c.f, c.dh, c.dy, stream=c.stream, **c.parts())
    assert got is grads and set(got) == {"gate", "pre_bias"}
    for k, old in (("gate", 2.0), ("pre_bias", -1.0)):
        v, tol = want[k]
        assert_close(k, grads[k], (v + old, tol + 2.0 ** -23 * (v.abs() + 3.0)))


def test_results_in_place():
    """y over x, dx over dy: the same bits as into other tensors."""
    for stream in (torch.bfloat16, torch.float32):
        c = Case(300, 192, stream, samples=3)
        x, f, p = c.x.to(DEV), c.f.to(DEV), c.parts(DEV)
        y, h = capi.block_norm(x, f, **p)
        dh, dy = c.dh.to(DEV), c.dy.to(DEV)
        dx, df, g = capi.block_norm_bwd(x, f, dh=dh, dy=dy, **p)
        dx2, df2, g2 = capi.block_norm_bwd(x, f, dh=dh, dy=dy, dx=dy, **p)
        y2, h2 = capi.block_norm(x, f, y=x, **p)
        assert dx2 is dy and y2 is x
        assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(dx, dx2) and torch.equal(df, df2)
        assert all(torch.equal(g[k], g2[k]) for k in g)


def test_surroundings_stay():
    T, C = 37, 136
    c = Case(T, C)
    p, x, f = c.parts(DEV), c.x.to(DEV), c.f.to(DEV)
    room = [torch.full((T + 2, C), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    y, h, dx, df = (r[1:-1] for r in room)
    capi.block_norm(x, f, y=y, h=h, **p)
    params = torch.full((7, C), 5.0, device=DEV)
    names = ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate")
    need = capi.swin_wattn_block_norm_bwd_workspace_bytes(T, C)
    ws = torch.full((need + 512,), 3, dtype=torch.uint8, device=DEV)
    capi.block_norm_bwd(x, f, dh=c.dh.to(DEV), dy=c.dy.to(DEV), dx=dx, df=df, grads=dict(zip(names, params[1:6])),
                        workspace=ws[256:256 + need], **p)
    torch.cuda.synchronize()
    for r in room:
        assert (r[0] == 7).all() and (r[-1] == 7).all() and (r[1:-1] != 7).any()
    assert (params[0] == 5).all() and (params[6] == 5).all()
    assert (ws[:256] == 3).all() and (ws[256 + need:] == 3).all()


def test_large_means_and_constant_rows():
    """A mean of 1000 spreads, and rows without any spread: their h is the bias."""
    c = Case(40, 512, stream=torch.float32, block=False, dy=1)
    c.x = torch.randn(40, 512, generator=torch.Generator().manual_seed(5)) + 1000.0
    c.check_forward()
    c.x[7] = 3.25
    c.x[8] = 0.0
    _, h = c.check_forward()
    assert torch.equal(h[7].cpu(), c.pre[1].bfloat16()) and torch.equal(h[8].cpu(), c.pre[1].bfloat16())


def test_nan_and_infinity_stay_in_their_token():
    c = Case(50, 96, samples=5)
    clean = capi.block_norm(c.x.to(DEV), c.f.to(DEV), **c.parts(DEV))
    clean_b = capi.block_norm_bwd(c.x.to(DEV), c.f.to(DEV), dh=c.dh.to(DEV), dy=c.dy.to(DEV), **c.parts(DEV))
    c.x[3, 5], c.f[11, 0], c.x[20, 95] = float("nan"), float("inf"), float("-inf")
    y, h = capi.block_norm(c.x.to(DEV), c.f.to(DEV), **c.parts(DEV))
    bad = torch.zeros(50, dtype=torch.bool)
    bad[[3, 11, 20]] = True
    assert torch.equal(y[~bad], clean[0][~bad]) and torch.equal(h[~bad], clean[1][~bad])
    assert all(torch.isnan(h[i]).any() for i in (3, 11, 20))
    dx, df, g = capi.block_norm_bwd(c.x.to(DEV), c.f.to(DEV), dh=c.dh.to(DEV), dy=c.dy.to(DEV), **c.parts(DEV))
    assert torch.equal(dx[~bad], clean_b[0][~bad]) and torch.equal(df[~bad], clean_b[1][~bad])
    assert torch.isnan(g["pre_weight"]).any()


def test_alpha_is_not_used_without_f():
    """Of the C entries, whose forward without f is h = pre(x) whatever alpha says."""
    c = Case(20, 96, block=False)
    lib, p = capi.load(), c.parts(DEV)
    x, dh, dy = c.x.to(DEV), c.dh.to(DEV), c.dy.to(DEV)
    h, dx = torch.empty_like(x), torch.empty_like(x)
    w, b = p["pre"]
    n, stream = None, torch.cuda.current_stream().cuda_stream
    ws = torch.empty(capi.swin_wattn_block_norm_bwd_workspace_bytes(20, 96), dtype=torch.uint8, device=DEV)
    at = lambda t: t.data_ptr()
    assert lib.swin_wattn_block_norm(at(x), n, at(w), at(b), n, n, n, n, n, at(h), 20, 96, 0, capi.BF16, capi.NORM_LAYER, -2.5, 1e-5,
                                     stream) == capi.OK
    assert lib.swin_wattn_block_norm_bwd(at(x), n, at(dh), at(dy), at(w), n, n, n, n, at(dx), n, n, n, n, n, n, 20, 96, 0, capi.BF16,
                                         capi.NORM_LAYER, -2.5, 1e-5, 0, at(ws), ws.numel(), stream) == capi.OK
    torch.cuda.synchronize()
    assert torch.equal(h, capi.block_norm(x, pre=p["pre"])[1])
    assert torch.equal(dx, capi.block_norm_bwd(x, dh=dh, dy=dy, pre=p["pre"])[0])


def test_no_tokens():
    c = Case(1, 96)
    e = torch.empty(0, 96, dtype=torch.bfloat16, device=DEV)
    y, h = capi.block_norm(e, e, **c.parts(DEV))
    assert y.shape == h.shape == (0, 96)
    dx, df, grads = capi.block_norm_bwd(e, e, dh=e, dy=e, **c.parts(DEV))
    assert all((g == 0).all() for g in grads.values()) and len(grads) == 5
    for g in grads.values():
        g.fill_(2.0)
    capi.block_norm_bwd(e, e, dh=e, dy=e, grads=grads, accumulate=True, **c.parts(DEV))
    assert all((g == 2).all() for g in grads.values())


def test_same_bits_on_every_run_and_other_stream():
    c = Case(3000, 192, samples=3)
    args = (c.x.to(DEV), c.f.to(DEV))
    kw = dict(dh=c.dh.to(DEV), dy=c.dy.to(DEV), **c.parts(DEV))
    a = capi.block_norm_bwd(*args, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = capi.block_norm_bwd(*args, stream=s, **kw)
    y, h = capi.block_norm(*args, stream=s, **c.parts(DEV))
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])
    y1, h1 = capi.block_norm(*args, **c.parts(DEV))
    assert torch.equal(y, y1) and torch.equal(h, h1)


def test_captured_and_replayed():
    c = Case(500, 384, samples=2)
    x, f, dh, dy, p = c.x.to(DEV), c.f.to(DEV), c.dh.to(DEV), c.dy.to(DEV), c.parts(DEV)
    y, h = torch.empty_like(x), torch.empty_like(f)
    dx, df = torch.empty_like(x), torch.empty_like(f)
    ws = torch.empty(capi.swin_wattn_block_norm_bwd_workspace_bytes(500, 384), dtype=torch.uint8, device=DEV)
    grads = {k: torch.empty(384, device=DEV) for k in ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate")}

    def step():
        capi.block_norm(x, f, y=y, h=h, **p)
        capi.block_norm_bwd(y, f, dh=dh, dy=dy, dx=dx, df=df, grads=grads, workspace=ws, **p)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn(500, 384).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, h, dx, df, *grads.values())]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, h, dx, df, *grads.values())))


def test_gradients_against_differences():
    """The gradients as differences of the forward itself: of a weighted sum of y and h in fp64, along
    random directions of every input, by the plain form whose values the kernels have been held to."""
    c = Case(12, 64, torch.float32, samples=3)
    dx, df, grads = capi.block_norm_bwd(*(t.to(DEV) for t in (forward64(c.x, c.f, stream=c.stream, **c.parts())[0][0].float(), c.f)),
                                        dh=c.dh.to(DEV), dy=c.dy.to(DEV), **c.parts(DEV))
    g = torch.Generator().manual_seed(3)

    def loss(step, name):
        p = {k: v for k, v in c.parts().items()}
        x, f = c.x.double(), c.f.double()
        if name == "x":
            x = x + step
        elif name == "f":
            f = f + step
        elif name == "gate":
            p["gate"] = p["gate"].double() + step
        else:
            where, what = name.split("_")
            w, b = p[where]
            p[where] = (w.double() + step, b) if what == "weight" else (w, b.double() + step)
        (y, _), (h, _) = forward64(x, f, stream=c.stream, **p)
        return float((y * c.dy.double()).sum() + (h * c.dh.double()).sum())

    for name, got in [("x", dx), ("f", df), *grads.items()]:
        dirn = torch.randn(got.shape, generator=g, dtype=torch.float64)
        eps = 1e-5
        want = (loss(eps * dirn, name) - loss(-eps * dirn, name)) / (2 * eps)
        have = float((got.double().cpu() * dirn).sum())
        # 2^-8 of each term for the roundings of df, and the differences' own error
        tol = 2.0 ** -8 * float((got.double().cpu() * dirn).square().sum().sqrt()) * 4 + 1e-7
        assert abs(want - have) <= tol, (name, want, have, tol)


def test_refusals():
    c = Case(8, 64)
    x, f, p = c.x.to(DEV), c.f.to(DEV), c.parts(DEV)
    good = dict(p)
    for bad in (dict(keep=torch.ones(3, device=DEV)), dict(gate=torch.ones(63, device=DEV)), dict(kind="batch"),
                dict(pre=(torch.ones(64, device=DEV).bfloat16(), None)), dict(y=torch.empty(8, 64, device=DEV))):
        with pytest.raises(ValueError):
            capi.block_norm(x, f, **{**good, **bad})
    with pytest.raises(ValueError):
        capi.block_norm(x[:, ::2], None, pre=(torch.ones(32, device=DEV), None))
    with pytest.raises(ValueError):
        capi.block_norm(x)
    with pytest.raises(ValueError):
        capi.block_norm(x, None, pre=p["pre"], gate=p["gate"])
    with pytest.raises(capi.SwinWAttnError) as e:
        capi.block_norm(x[:, :60].contiguous(), None, pre=(torch.ones(60, device=DEV), None))
    assert e.value.status == capi.ERR_UNSUPPORTED
    with pytest.raises(capi.SwinWAttnError) as e:
        capi.block_norm(x, f, **{**good, "eps": 0.0})
    assert e.value.status == capi.ERR_INVALID_ARG
    with pytest.raises(capi.SwinWAttnError) as e:  # h over f
        capi.block_norm(x, f, h=f, **good)
    assert e.value.status == capi.ERR_INVALID_ARG
    odd = torch.empty(8 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(8, 64)
    with pytest.raises(capi.SwinWAttnError) as e:
        capi.block_norm(odd, f, **good)
    assert e.value.status == capi.ERR_MISALIGNED
    with pytest.raises(ValueError):
        capi.block_norm_bwd(x, f, dh=None, dy=None, **{**good, "pre": None})
    with pytest.raises(ValueError):
        capi.block_norm_bwd(x, f, dh=None, **good)
    with pytest.raises(ValueError):
        capi.block_norm_bwd(x, f, dh=f, grads={"gate": torch.ones(64, device=DEV)}, **{**good, "gate": None})
    with pytest.raises(capi.SwinWAttnError):
        capi.block_norm_bwd(x, f, dh=c.dh.to(DEV), workspace=torch.empty(256, dtype=torch.uint8, device=DEV), **good)
