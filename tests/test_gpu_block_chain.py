"""The operators around a block's products run together as they are used: a training step of a block's MLP
half (norm, products, residual with gate and stochastic depth, all gradients, clipping, weight updates), and the
same half served on 4-bit operands; and each operator at offsets that pass 32 bits, from several threads and
on shared streams."""
import threading

import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.block_norm_util import assert_close, forward64
from tests.fp4_util import quantize64
from tests.linear_util import assert_within
from tests.test_gpu_fp4 import linear64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _rand(seed, *shape, std=1.0, dtype=torch.bfloat16, mean=0.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std + mean).to(dtype)


def test_training_step():
    """x -> h = norm(x) -> f = fc2(gelu(fc1 h)) -> y = x + keep gate f, g = norm2(y): gradients of all parameters and of x for
    given gradients of y and g, clipped, and the weight updates. Each intermediate is rounded to bf16 (2^-9 of its
    root mean square, four of them on the way to a gradient): a hundredth in the 2-norm holds them all."""
    T, C, S = 300, 192, 3
    x = _rand(1, T, C)
    n1, n2 = [(_rand(s, C, std=0.2, mean=1.0, dtype=torch.float32), _rand(s + 1, C, std=0.2, dtype=torch.float32)) for s in (2, 4)]
    gate, keep = _rand(6, C, std=0.3, mean=0.7, dtype=torch.float32), torch.tensor([1.25, 0.0, 1.25])
    w1, w2 = _rand(7, 4 * C, C, std=C ** -0.5), _rand(8, C, 4 * C, std=(4 * C) ** -0.5)
    b1, b2 = _rand(9, 4 * C, std=0.1, dtype=torch.float32), _rand(10, C, std=0.1, dtype=torch.float32)
    dy, dg = _rand(11, T, C, std=1e-2), _rand(12, T, C, std=1e-2)
    to = lambda *ts: [t.to(DEV) for t in ts]
    xd, gd, kd, w1d, w2d, b1d, b2d, dyd, dgd = to(x, gate, keep, w1, w2, b1, b2, dy, dg)
    n1d, n2d = tuple(to(*n1)), tuple(to(*n2))

    def step(out):
        _, h = capi.block_norm(xd, pre=n1d)
        pre = torch.empty(T, 4 * C, dtype=torch.bfloat16, device=DEV)
        a = capi.linear(h, w1d, b1d, act="gelu", pre=pre)
        f = capi.linear(a, w2d, b2d)
        y, g = capi.block_norm(xd, f, pre=n2d, gate=gd, keep=kd)
        dx, df, ng2 = capi.block_norm_bwd(y, f, dh=dgd, dy=dyd, pre=n2d, gate=gd, keep=kd)
        dw2, db2 = capi.linear_bwd_weight(df, a)
        dpre = capi.linear_bwd_data(df, w2d, pre=pre, act="gelu")
        dw1, db1 = capi.linear_bwd_weight(dpre, h)
        dh = capi.linear_bwd_data(dpre, w1d)
        dx, _, ng1 = capi.block_norm_bwd(xd, dh=dh, dy=dx, pre=n1d, dx=dx)
        grads = [dw1, dw2, db1, db2, ng1["pre_weight"], ng1["pre_bias"], ng2["pre_weight"], ng2["pre_bias"], ng2["gate"]]
        raw = [t.clone() for t in grads]
        norm = capi.GradClip(grads)(0.05)
        out.update(y=y, g=g, dx=dx, raw=raw, clipped=grads, norm=norm, update=[capi.orthogonalize(w) for w in grads[:2]])

    got = {}
    step(got)
    torch.cuda.synchronize()

    leaf = lambda t: t.double().requires_grad_(True)
    x64, w1l, w2l, b1l, b2l, gl = map(leaf, (x, w1, w2, b1, b2, gate))
    m1, m2 = [tuple(map(leaf, n)) for n in (n1, n2)]
    norm = lambda v, wb: torch.nn.functional.layer_norm(v, (C,), wb[0], wb[1], 1e-5)
    f64 = torch.nn.functional.gelu(norm(x64, m1) @ w1l.T + b1l) @ w2l.T + b2l
    y64 = x64 + keep.double().repeat_interleave(T // S)[:, None] * gl * f64
    g64 = norm(y64, m2)
    leaves = (w1l, w2l, b1l, b2l, *m1, *m2, gl)
    ref = torch.autograd.grad([y64, g64], [x64, *leaves], [dy.double(), dg.double()])
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())
    assert rel(got["y"], y64.detach()) < 1e-2 and rel(got["g"], g64.detach()) < 1e-2 and rel(got["dx"], ref[0]) < 1e-2
    for a, b in zip(got["raw"], ref[1:]):
        assert rel(a, b) < 1e-2
    # the clipping of these gradients, to the accuracy of its own test
    n = sum(float(t.double().square().sum()) for t in got["raw"]) ** 0.5
    assert abs(float(got["norm"]) - n) < 1e-6 * n and n > 0.05
    for a, b in zip(got["clipped"], got["raw"]):
        assert torch.allclose(a.double(), b.double() * (0.05 / (n + 1e-6)), rtol=2e-6, atol=0)
    for u in got["update"]:
        s = torch.linalg.svdvals(u.float())
        assert 0.6 < float(s[0]) < 1.3
    # the same bits again
    again = {}
    step(again)
    assert torch.equal(got["dx"], again["dx"]) and torch.equal(got["norm"], again["norm"])
    assert all(torch.equal(a, b) for a, b in zip(got["clipped"] + got["update"], again["clipped"] + again["update"]))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 49, 777])
def test_served_on_4_bit_operands(fmt, T):
    """norm -> fc1 with GELU -> fc2 with the shortcut, weights quantised once: every step held to its own bound on the
    step before it."""
    C = 384
    x, wb = _rand(T, T, C), (_rand(2, C, std=0.2, mean=1.0, dtype=torch.float32), _rand(3, C, std=0.2, dtype=torch.float32))
    w1, w2 = _rand(4, 4 * C, C, std=C ** -0.5), _rand(5, C, 4 * C, std=(4 * C) ** -0.5)
    b1, b2 = _rand(6, 4 * C, std=0.1, dtype=torch.float32), _rand(7, C, std=0.1, dtype=torch.float32)
    q1, q2 = (capi.quantize_fp4(w.to(DEV), fmt) for w in (w1, w2))
    scales = [torch.full((1,), 2.0 ** -e, device=DEV) if fmt == "nvfp4" else None for e in (9, 8)]
    xd = x.to(DEV)
    _, h = capi.block_norm(xd, pre=tuple(t.to(DEV) for t in wb))
    a = capi.linear_fp4(h, q1, b1.to(DEV), act="gelu", x_scale=scales[0])
    y = capi.linear_fp4(a, q2, b2.to(DEV), residual=xd, x_scale=scales[1])
    torch.cuda.synchronize()
    _, want = forward64(x, None, wb, None, None, None, 1.0, "layer", 1e-5, torch.bfloat16)
    assert_close("h", h, want)
    decoded = [capi.dequantize_fp4(q, torch.float32).double().cpu() for q in (q1, q2)]
    values = lambda t, s: quantize64(t.cpu(), fmt, None if s is None else float(s))[2]
    assert_within("a", a, *linear64(values(h, scales[0]), decoded[0], b1, "gelu", None))
    assert_within("y", y, *linear64(values(a, scales[1]), decoded[1], b2, "none", x))


# ---- offsets that pass 32 bits -------------------------------------------------------

def _rows(n):
    """Rows at both ends and around the elements 2^31 and 2^32 of 8192 a row."""
    at = [0, 1, n - 2, n - 1, *(r + d for r in (2 ** 31 // 8192, 2 ** 32 // 8192) for d in (-1, 0, 1))]
    return torch.tensor(sorted({r for r in at if 0 <= r < n}))


def _big(n, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(5)
    return torch.randn(n, 8192, generator=g, device=DEV, dtype=torch.bfloat16).to(dtype)


def test_walked_rows_past_32_bits():
    T, C = 2900000, 1536  # 4.5e9 elements, in the form that walks rows
    x = _big(T * C // 8192 + 1).view(-1)[:T * C].view(T, C)
    f = x.roll(1, 0)
    wb = (_rand(2, C, std=0.2, mean=1.0, dtype=torch.float32), _rand(3, C, std=0.2, dtype=torch.float32))
    wbd, keep = tuple(t.to(DEV) for t in wb), (torch.arange(T, device=DEV) % 5).float()
    r = torch.tensor(sorted({q for b in (0, 2 ** 31 // C, 2 ** 32 // C, T - 1) for q in (b - 1, b, b + 1) if 0 <= q < T}), device=DEV)
    pick = lambda t: t[r].cpu()
    xs, fs, ks = pick(x), pick(f), pick(keep)
    y, h = capi.block_norm(x, f, pre=wbd, post=wbd, keep=keep, y=x)
    want_y, want_h = forward64(xs, fs, wb, wb, None, ks, 1.0, "layer", 1e-5, torch.bfloat16)
    assert_close("y", pick(y), want_y)
    assert_close("h", pick(h), want_h)



def test_norms_past_32_bits():
    T, C = 530000, 8192  # 4.3e9 elements
    x, f = _big(T), _big(T)
    wb = (_rand(2, C, std=0.2, mean=1.0, dtype=torch.float32), _rand(3, C, std=0.2, dtype=torch.float32))
    wbd = tuple(t.to(DEV) for t in wb)
    y, h = capi.block_norm(x, f, pre=wbd, y=x)  # in place
    r = _rows(T)
    xs = _big(T)
    want_y, want_h = forward64(xs[r.to(DEV)].cpu(), f[r.to(DEV)].cpu(), wb, None, None, None, 1.0, "layer", 1e-5, torch.bfloat16)
    assert_close("y", y[r.to(DEV)], want_y)
    assert_close("h", h[r.to(DEV)], want_h)
    from tests.block_norm_util import backward64
    dx, df, grads = capi.block_norm_bwd(xs, f, dh=f, pre=wbd, dx=y, df=h)
    pick = lambda t: t[r.to(DEV)].cpu()
    want = backward64(pick(xs), pick(f), pick(f), None, wb, None, None, None, 1.0, "layer", 1e-5, torch.bfloat16)
    assert_close("dx", pick(dx), want["dx"])
    assert_close("df", pick(df), want["df"])
    # the sum of dh, 530000 values of one sign at random each: within 1e-3 of their spread
    ref = torch.zeros(C, dtype=torch.float64, device=DEV)
    for part in f.split(20000):
        ref += part.double().sum(0)
    assert float((grads["pre_bias"].double() - ref).abs().max()) < 1e-3 * T ** 0.5


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_4_bit_operands_past_32_bits(fmt):
    T = 530000
    x = _big(T)
    q = capi.quantize_fp4(x, fmt)
    back = capi.dequantize_fp4(q)
    r = _rows(T).to(DEV)
    ts = None if fmt == "mxfp4" else float(q.tensor_scale)
    assert ts is None or ts == 2.0 ** -9 or ts == 2.0 ** -8
    assert torch.equal(back[r].double().cpu(), quantize64(x[r].cpu(), fmt, ts)[2])
    del x, back
    # a product whose result passes 2^32 elements, of a narrow K, and one of this wide x
    xs = _rand(1, T, 32).to(DEV)
    w = _rand(2, 8192, 32)
    wq = capi.quantize_fp4(w.to(DEV), fmt)
    y = capi.linear_fp4(xs, wq)
    xv = capi.dequantize_fp4(capi.quantize_fp4(xs, fmt), torch.float32)[r].double().cpu()
    wv = capi.dequantize_fp4(wq, torch.float32).double().cpu()
    assert_within("y", y[r], *linear64(xv, wv, None, "none", None))
    del y
    wide = capi.quantize_fp4(_rand(3, 24, 8192).to(DEV), fmt)
    y = capi.linear_fp4(q, wide)
    pick = lambda t: capi.dequantize_fp4(t, torch.float32)
    xv = quantize64(_big(T)[r].cpu(), fmt, ts)[2]
    assert_within("y", y[r], *linear64(xv, pick(wide).double().cpu(), None, "none", None))


def test_clipping_past_32_bits():
    g = torch.full((4300000001,), 1e-3, dtype=torch.bfloat16, device=DEV)
    v = float(g[0])
    small = torch.full((5,), 2.0, device=DEV)
    n = capi.GradClip([g, small])(1.0)
    torch.cuda.synchronize()
    want = (g.numel() * v * v + 20.0) ** 0.5
    assert abs(float(n) - want) < 1e-6 * want
    c = torch.tensor(v * (1.0 / (want + 1e-6)), dtype=torch.float64)
    for at in (0, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, g.numel() - 1):
        assert abs(float(g[at]) - float(c)) <= 2.0 ** -8 * float(c) * 1.01
    assert torch.allclose(small.double().cpu(), 2.0 / torch.tensor(want + 1e-6).double(), rtol=1e-6)


# ---- several threads -----------------------------------------------------------------

def test_several_threads_and_streams():
    """Calls from four threads on a stream each, at once: the results of one at a time."""
    T, C = 500, 384
    x, f = _rand(1, T, C).to(DEV), _rand(2, T, C).to(DEV)
    wb = tuple(t.to(DEV) for t in (_rand(3, C, mean=1.0, dtype=torch.float32), _rand(4, C, dtype=torch.float32)))
    wq = capi.quantize_fp4(_rand(5, 768, C).to(DEV), "nvfp4")
    grads = [_rand(6 + i, 4000 + i, dtype=torch.float32).to(DEV) for i in range(20)]

    def work(stream):
        y, h = capi.block_norm(x, f, pre=wb, stream=stream)
        dx, df, g = capi.block_norm_bwd(y, f, dh=h, dy=y, pre=wb, stream=stream)
        z = capi.linear_fp4(h, wq, stream=stream)
        with torch.cuda.stream(stream):
            out = [torch.empty_like(t) for t in grads]
        n = capi.GradClip(grads, out=out)(0.5, stream=stream)
        return [y, h, dx, df, z, n, *g.values(), *out]

    torch.cuda.synchronize()
    first = torch.cuda.Stream()
    want = work(first)
    first.synchronize()
    results, errors = {}, []

    def run(k):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got = work(s)
            s.synchronize()
            results[k] = got
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for got in results.values():
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_launch_counts():
    x = _rand(1, 300, 192).to(DEV)
    wb = tuple(t.to(DEV) for t in (_rand(3, 192, mean=1.0, dtype=torch.float32), _rand(4, 192, dtype=torch.float32)))
    w, g = capi.quantize_fp4(_rand(5, 64, 192).to(DEV), "nvfp4"), torch.ones(10, device=DEV)
    clip = capi.GradClip([g])
    scale = torch.full((1,), 2.0 ** -9, device=DEV)
    for want, call in ((1, lambda: capi.block_norm(x, pre=wb)), (2, lambda: capi.block_norm_bwd(x, dh=x, pre=wb)),
                       (1, lambda: capi.block_norm_bwd(x, dh=x, pre=wb, grads={})), (2, lambda: clip(1.0)),
                       (2, lambda: capi.quantize_fp4(x)), (1, lambda: capi.quantize_fp4(x, "mxfp4")), (1, lambda: capi.dequantize_fp4(w)),
                       (3, lambda: capi.linear_fp4(x, w)), (2, lambda: capi.linear_fp4(x, w, x_scale=scale)),
                       (1, lambda: capi.linear_fp4(x[:3], w, x_scale=scale))):
        capi.swin_wattn_launch_count(reset=True)
        call()
        assert capi.swin_wattn_launch_count() == want
