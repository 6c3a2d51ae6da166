"""The MLP's products and their gradients on the GPU against plain fp64 forms, through the
public entry points: ragged token counts from one, widths of one chunk and many, every
activation, integer inputs whose results are exact, results over their own second operand,
untouched surroundings, accumulation, other streams, graph replays and the error paths."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.linear_util import (ACTS, act64, assert_within, bwd_data64, bwd_weight64, linear64, slope64)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _rand(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _ints(seed, *shape, hi=3):
    """Small whole numbers: products and sums of them are exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-hi, hi + 1, shape, generator=g).to(torch.bfloat16)


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _ok(status):
    torch.cuda.synchronize()
    assert int(status.item()) == 0


SIZES = [  # tokens, K, N
    (1, 8, 8), (1, 1536, 1000), (2, 64, 40), (7, 96, 384), (17, 136, 264), (49, 1536, 512), (64, 64, 64),
    (100, 384, 1152), (127, 72, 32), (128, 128, 256), (129, 200, 1000), (255, 512, 96), (257, 2048, 72),
    (300, 40, 2000), (777, 384, 136), (1000, 192, 768), (4099, 96, 384), (20000, 32, 48), (2100, 512, 2048),
]


@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear_exact_on_whole_numbers(T, K, N):
    """Every result is a whole number below 2^24 before its one rounding, so it is known to
    the bit: a row, column or chunk read twice, left out or misplaced shows."""
    x, w = _ints(T + K, T, K), _ints(N, N, K, hi=2)
    b = _ints(3, N, hi=9).float()
    r = _ints(4, T, N, hi=50)
    xd, wd, bd, rd = _dev(x, w, b, r)
    z = x.double() @ w.double().T
    st = _status()
    y = capi.linear(xd, wd, status=st)
    pre = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    y2 = capi.linear(xd, wd, bd, act="relu", residual=rd, pre=pre, status=st)
    _ok(st)
    assert torch.equal(y.cpu(), z.to(torch.bfloat16))
    zb = z + b.double()
    assert torch.equal(pre.cpu(), zb.to(torch.bfloat16))
    assert torch.equal(y2.cpu(), (zb.clamp_min(0) + r.double()).to(torch.bfloat16))


@pytest.mark.parametrize("T,K,N", SIZES)
def test_gradients_exact_on_whole_numbers(T, K, N):
    dy, x, w, pre = _ints(T, T, N), _ints(K, T, K), _ints(N, N, K, hi=2), _ints(5, T, K)
    dyd, xd, wd, pd = _dev(dy, x, w, pre)
    st = _status()
    dx = capi.linear_bwd_data(dyd, wd, status=st)
    dxr = capi.linear_bwd_data(dyd, wd, pre=pd, act="relu", status=st)
    dw, db = capi.linear_bwd_weight(dyd, xd, status=st)
    dw16 = torch.full((N, K), 3.0, dtype=torch.bfloat16, device=DEV)
    _, none = capi.linear_bwd_weight(dyd, xd, dw=dw16, status=st)
    _ok(st)
    d = dy.double() @ w.double()
    assert none is None
    assert torch.equal(dx.cpu(), d.to(torch.bfloat16))
    assert torch.equal(dxr.cpu().double(), torch.where(pre > 0, d, torch.zeros_like(d)).to(torch.bfloat16).double())
    g = dy.double().T @ x.double()
    assert torch.equal(dw.cpu().double(), g)
    assert torch.equal(db.cpu().double(), dy.double().sum(0))
    assert torch.equal(dw16.cpu(), g.to(torch.bfloat16))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", [(1, 200, 120), (50, 384, 1536), (333, 128, 264), (1500, 64, 96)])
def test_linear_against_fp64(T, K, N, act):
    x, w, b = _rand(T, T, K), _rand(1, N, K, std=2.0 * K ** -0.5), _rand(2, N, dtype=torch.float32)
    r = _rand(3, T, N)
    xd, wd, bd, rd = _dev(x, w, b, r)
    pre = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    st = _status()
    for bias, res in ((b, None), (b, r), (None, r), (None, None)):
        y = capi.linear(xd, wd, None if bias is None else bd, act=act, residual=None if res is None else rd, pre=pre,
                        status=st)
        _ok(st)
        yr, zr, ytol, ztol = linear64(x, w, bias, act, res)
        assert_within("y", y, yr, ytol)
        assert_within("pre", pre, zr, ztol)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", [(1, 200, 120), (50, 384, 1536), (333, 128, 264), (1500, 64, 96)])
def test_bwd_data_against_fp64(T, K, N, act):
    dy, w, pre = _rand(T, T, N, std=1e-2), _rand(1, N, K, std=K ** -0.5), _rand(2, T, K, std=2.0)
    st = _status()
    dx = capi.linear_bwd_data(*_dev(dy, w), pre=pre.to(DEV), act=act, status=st)
    _ok(st)
    ref, tol = bwd_data64(dy, w, pre, act)
    assert_within("dx", dx, ref, tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K,N", [(1, 96, 200), (63, 64, 64), (500, 136, 264), (5000, 48, 104), (3001, 1536, 520)])
def test_bwd_weight_against_fp64_and_accumulates(T, K, N, dtype):
    dy, x = _rand(T, T, N, std=1e-2), _rand(1, T, K)
    dyd, xd = _dev(dy, x)
    dw = torch.empty(N, K, dtype=dtype, device=DEV)
    db = torch.empty(N, device=DEV)
    st = _status()
    capi.linear_bwd_weight(dyd, xd, dw=dw, db=db, status=st)
    _ok(st)
    rw, rb, tw, tb = bwd_weight64(dy, x, dtype)
    assert_within("dw", dw, rw, tw)
    assert_within("db", db, rb, tb)
    old_w, old_b = _rand(2, N, K, dtype=dtype), _rand(3, N, dtype=torch.float32)
    dw.copy_(old_w)
    db.copy_(old_b)
    capi.linear_bwd_weight(dyd, xd, dw=dw, db=db, accumulate=True, status=st)
    _ok(st)
    rw, rb, tw, tb = bwd_weight64(dy, x, dtype, old_w, old_b)
    assert_within("accumulated dw", dw, rw, tw)
    assert_within("accumulated db", db, rb, tb)


@pytest.mark.parametrize("act", ACTS[1:])
def test_activation_over_the_whole_line(act):
    """act and act' of every finite bf16 value (through an identity weight), and of the
    special ones: NaN stays NaN, +inf gives +inf and slope 1, -inf (and the far tail) 0."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16).reshape(-1, 8)
    v = torch.where(v.abs() < 1e30, v, torch.zeros_like(v))
    vd = v.to(DEV)
    eye = torch.eye(8, dtype=torch.bfloat16, device=DEV)
    y = capi.linear(vd, eye, act=act)
    torch.cuda.synchronize()
    ref = act64(v.double(), act)
    ref = torch.where(v.double() < -1e3, torch.zeros_like(ref), ref)  # 0 * huge is 0, not NaN
    # the tail keeps its relative accuracy: GELU's fit to 5e-5 down to z = -6 (6e-9 in size
    # there); the exponent of the others, up to 127, is off by a few 2^-24 of itself
    tail = 6e-5 * ref.abs() + 1e-30 if act == "gelu" else 3e-5 * ref.abs() + 1e-30
    if act == "gelu":
        tail = tail + torch.where(v < -6.0, 1e-8, 0.0).double()
    tol = torch.minimum(torch.full_like(ref, 7.5e-6), tail) + 2.0 ** -8 * ref.abs()
    assert_within(act, y, ref, tol)
    one = torch.ones(v.shape[0], 8, dtype=torch.bfloat16, device=DEV)
    dx = capi.linear_bwd_data(one, eye, pre=vd, act=act)
    torch.cuda.synchronize()
    near = v.double().clamp(-1e3, 1e3)
    ref = slope64(near, act)
    ref = torch.where(torch.isnan(ref), torch.zeros_like(ref), ref)
    assert_within(act + "'", dx, ref, 3e-5 + 2.0 ** -8 * ref.abs())
    sp = torch.tensor([[float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 200.0, -200.0, 1.0]],
                      dtype=torch.bfloat16, device=DEV)
    dx = capi.linear_bwd_data(torch.ones_like(sp), eye, pre=sp, act=act).float().cpu()[0]
    assert (torch.isnan(dx[0]) if act != "relu" else dx[0] == 0) and dx[1] == 1 and dx[2].abs() < 1e-29
    assert dx[5] == 1 and dx[6].abs() < 1e-29
    # a non-finite value reaches every column of its own row, and no other row
    x = torch.ones(3, 8, dtype=torch.bfloat16, device=DEV)
    x[1, 2] = float("nan")
    yn = capi.linear(x, torch.ones(16, 8, dtype=torch.bfloat16, device=DEV), act=act).float()
    assert torch.isnan(yn[1]).all() and torch.isfinite(yn[0]).all() and torch.isfinite(yn[2]).all()
    x[1, 2] = float("inf")
    yn = capi.linear(x, torch.ones(16, 8, dtype=torch.bfloat16, device=DEV), act=act).float()
    assert torch.isinf(yn[1]).all() and torch.isfinite(yn[0]).all()


def test_results_over_their_second_operand_and_untouched_surroundings():
    T, K, N = 301, 96, 200
    x, w, b, r = _rand(1, T, K), _rand(2, N, K, std=0.1), _rand(3, N, dtype=torch.float32), _rand(4, T, N)
    xd, wd, bd, rd = _dev(x, w, b, r)
    y = capi.linear(xd, wd, bd, act="gelu", residual=rd)
    buf = torch.full((T * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    inplace = buf[32:32 + T * N].view(T, N)
    inplace.copy_(rd)
    assert capi.linear(xd, wd, bd, act="gelu", residual=inplace, y=inplace) is inplace
    torch.cuda.synchronize()
    assert torch.equal(inplace, y)
    assert torch.all(buf[:32] == 7.0) and torch.all(buf[32 + T * N:] == 7.0)
    dy, pre = _rand(5, T, N), _rand(6, T, K)
    dyd, pd = _dev(dy, pre)
    dx = capi.linear_bwd_data(dyd, wd, pre=pd, act="silu")
    over = pd.clone()
    capi.linear_bwd_data(dyd, wd, pre=over, act="silu", dx=over)
    buf = torch.full((N * K + 64,), 7.0, device=DEV)
    dw = buf[32:32 + N * K].view(N, K)
    capi.linear_bwd_weight(dyd, xd, dw=dw)
    torch.cuda.synchronize()
    assert torch.equal(over, dx)
    assert torch.all(buf[:32] == 7.0) and torch.all(buf[32 + N * K:] == 7.0)


def test_no_tokens():
    w = _rand(1, 64, 32).to(DEV)
    x = torch.empty(0, 32, dtype=torch.bfloat16, device=DEV)
    dy = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    assert capi.linear(x, w).shape == (0, 64)
    assert capi.linear_bwd_data(dy, w).shape == (0, 32)
    dw, db = capi.linear_bwd_weight(dy, x)
    torch.cuda.synchronize()
    assert torch.all(dw == 0) and torch.all(db == 0)
    dw.fill_(2.0)
    db.fill_(3.0)
    capi.linear_bwd_weight(dy, x, dw=dw, db=db, accumulate=True)
    torch.cuda.synchronize()
    assert torch.all(dw == 2.0) and torch.all(db == 3.0)


def test_leading_axes_and_one_dimension():
    x, w = _rand(1, 2, 3, 5, 64), _rand(2, 40, 64, std=0.1)
    xd, wd = _dev(x, w)
    y = capi.linear(xd, wd)
    assert y.shape == (2, 3, 5, 40)
    assert torch.equal(y.reshape(-1, 40), capi.linear(xd.reshape(-1, 64), wd))
    assert torch.equal(capi.linear(xd[1, 2, 4], wd), y[1, 2, 4])
    dx = capi.linear_bwd_data(y, wd)
    dw, db = capi.linear_bwd_weight(y, xd)
    assert dx.shape == x.shape and dw.shape == (40, 64) and db.shape == (40,)


def test_deterministic():
    dy, x, w = _rand(1, 9000, 96).to(DEV), _rand(2, 9000, 64).to(DEV), _rand(3, 96, 64).to(DEV)
    a, b = capi.linear_bwd_weight(dy, x), capi.linear_bwd_weight(dy, x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(capi.linear(x, w, act="gelu"), capi.linear(x, w, act="gelu"))


def test_two_streams_at_once():
    """Two calls of each kind in flight on two streams, with their own workspaces."""
    T, K, N = 6000, 128, 96
    data = [(_rand(s, T, N), _rand(s + 1, T, K), _rand(s + 2, N, K, std=0.1)) for s in (10, 20)]
    dev = [_dev(*d) for d in data]
    want = [(capi.linear(x, w, act="gelu"), capi.linear_bwd_data(dy, w), *capi.linear_bwd_weight(dy, x))
            for dy, x, w in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [(capi.linear(x, w, act="gelu", stream=s), capi.linear_bwd_data(dy, w, stream=s),
                *capi.linear_bwd_weight(dy, x, stream=s)) for (dy, x, w), s in zip(dev, streams)]
        torch.cuda.synchronize()
        for g, r in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, r))


def test_mlp_training_step_in_a_graph():
    """The operators as a block uses them, y = x + fc2(gelu(fc1(x))), forward, backward and
    the orthogonalised updates, captured once and replayed on new inputs: each result against
    the fp64 form on the kernels' own bf16 intermediates, and the chain against fp64
    differences."""
    T, C, H = 196, 64, 256
    x, dy = torch.empty(T, C, dtype=torch.bfloat16, device=DEV), torch.empty(T, C, dtype=torch.bfloat16, device=DEV)
    w1, w2 = _rand(1, H, C, std=C ** -0.5), _rand(2, C, H, std=H ** -0.5)
    b1, b2 = _rand(3, H, std=0.1, dtype=torch.float32), _rand(4, C, std=0.1, dtype=torch.float32)
    w1d, w2d, b1d, b2d = _dev(w1, w2, b1, b2)
    pre = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    st = _status()

    def step():
        h = capi.linear(x, w1d, b1d, act="gelu", pre=pre, status=st)
        y = capi.linear(h, w2d, b2d, residual=x, status=st)
        dpre = capi.linear_bwd_data(dy, w2d, pre=pre, act="gelu", status=st)
        dx = capi.linear_bwd_data(dpre, w1d, status=st)
        dw2, db2 = capi.linear_bwd_weight(dy, h, status=st)
        dw1, db1 = capi.linear_bwd_weight(dpre, x, status=st)
        return h, y, dpre, dx, dw2, db2, dw1, db1, capi.orthogonalize(dw1, status=st), capi.orthogonalize(dw2, status=st)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (50, 60):
        xs, dys = _rand(seed, T, C), _rand(seed + 1, T, C, std=1e-2)
        x.copy_(xs)
        dy.copy_(dys)
        graph.replay()
        _ok(st)
        h, y, dpre, dx, dw2, db2, dw1, db1, o1, o2 = [o.cpu() for o in outs]
        p = pre.cpu()
        for name, got, (ref, _, tol, _) in (("h", h, linear64(xs, w1, b1, "gelu", None)),
                                            ("y", y, linear64(h, w2, b2, "none", xs))):
            assert_within(name, got, ref, tol)
        assert_within("dpre", dpre, *bwd_data64(dys, w2, p, "gelu"))
        assert_within("dx", dx, *bwd_data64(dpre, w1, None, "none"))
        for name, gw, gb, a, b in (("2", dw2, db2, dys, h), ("1", dw1, db1, dpre, xs)):
            rw, rb, tw, tb = bwd_weight64(a, b, torch.float32)
            assert_within("dw" + name, gw, rw, tw)
            assert_within("db" + name, gb, rb, tb)
        for o, g in ((o1, dw1), (o2, dw2)):
            sv = torch.linalg.svdvals(o.double())
            gs = torch.linalg.svdvals(g.double())
            strong = gs > 0.05 * gs[0]
            assert float(sv.max()) < 1.25 and float(sv[:int(strong.sum())].min()) > 0.6
        # the loss sum(y dy) in fp64 against the chain's gradients, by central differences in
        # random directions. The chain's values carry four bf16 roundings (pre, h, dpre, dx),
        # each up to 2^-8 of its value, so the gradient is off by a vector of at most 4 * 2^-8 of
        # its norm; along a direction of independent N(0, 1) entries that is at most five
        # deviations of 4 * 2^-8 |gradient|.
        gen = torch.Generator().manual_seed(seed)

        def loss(xv, w1v, b1v, w2v, b2v):
            hh = act64(xv @ w1v.T + b1v, "gelu")
            return float((((hh @ w2v.T) + b2v) * dys.double()).sum())

        args = [t.double() for t in (xs, w1, b1, w2, b2)]
        grads = [dx, dw1, db1, dw2, db2]
        for i, gr in enumerate(grads):
            d = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
            eps = 1e-5
            up, dn = list(args), list(args)
            up[i], dn[i] = args[i] + eps * d, args[i] - eps * d
            fd = (loss(*up) - loss(*dn)) / (2 * eps)
            an = float((gr.double() * d).sum())
            assert abs(fd - an) <= 5 * 4 * 2.0 ** -8 * float(gr.double().norm()) + 1e-6, (i, fd, an)


def test_two_graphs_with_their_own_workspaces():
    T, K, N = 8000, 64, 96
    dy, x = [_rand(s, T, N).to(DEV) for s in (1, 2)], [_rand(s, T, K).to(DEV) for s in (3, 4)]
    want = [capi.linear_bwd_weight(a, b)[0].clone() for a, b in zip(dy, x)]
    graphs, outs = [], []
    for a, b in zip(dy, x):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(capi.linear_bwd_weight(a, b)[0])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_error_paths():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device=DEV)
    x, w, b, y = z(4, 96), z(64, 96), z(64, d=torch.float32), torch.full((4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    p = lambda t: None if t is None else t.data_ptr()

    def f(xp=x.data_ptr(), wp=w.data_ptr(), bp=b.data_ptr(), rp=None, yp=y.data_ptr(), pp=None, T=4, K=96, N=64, act=0,
          st=None):
        return capi.swin_wattn_linear(xp, wp, bp, rp, yp, pp, T, K, N, act, st, s)

    assert f(T=0) == capi.OK
    assert f(T=-1) == capi.ERR_INVALID_ARG and f(act=9) == capi.ERR_INVALID_ARG
    assert f(K=92) == capi.ERR_UNSUPPORTED and f(N=60) == capi.ERR_UNSUPPORTED and f(K=0) == capi.ERR_UNSUPPORTED
    assert f(K=32776) == capi.ERR_UNSUPPORTED
    assert f(yp=None) == capi.ERR_INVALID_ARG
    assert f(yp=x.data_ptr()) == capi.ERR_INVALID_ARG       # y over x
    assert f(pp=y.data_ptr()) == capi.ERR_INVALID_ARG       # pre over y
    assert f(rp=y.data_ptr() + 16) == capi.ERR_INVALID_ARG  # residual shifted against y
    assert f(xp=x.data_ptr() + 2) == capi.ERR_MISALIGNED
    assert f(xp=torch.zeros(4, 96, dtype=torch.bfloat16).data_ptr()) == capi.ERR_INVALID_ARG
    dw, db = z(64, 96, d=torch.float32), z(64, d=torch.float32)
    need = capi.swin_wattn_linear_bwd_weight_workspace_bytes(4, 96, 64)
    ws = torch.zeros(need + 256, dtype=torch.uint8, device=DEV)

    def h(wsp=ws.data_ptr(), nb=need, dtype=capi.FP32, dwp=dw.data_ptr(), dbp=db.data_ptr()):
        return capi.swin_wattn_linear_bwd_weight(y.data_ptr(), x.data_ptr(), dwp, dbp, 4, 96, 64, dtype, 0, wsp, nb,
                                                 None, s)

    assert h(nb=need - 1) == capi.ERR_INVALID_ARG and h(dtype=5) == capi.ERR_INVALID_ARG
    assert h(wsp=ws.data_ptr() + 16) == capi.ERR_MISALIGNED
    assert h(dbp=dw.data_ptr()) == capi.ERR_INVALID_ARG
    assert capi.swin_wattn_linear_bwd_data(y.data_ptr(), w.data_ptr(), None, x.data_ptr(), 4, 96, 64, capi.ACT_GELU,
                                           None, s) == capi.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.all(y == 3.0)
    with pytest.raises(ValueError):
        capi.linear(x.float(), w)
    with pytest.raises(ValueError):
        capi.linear(z(4, 192)[:, ::2], w)
    with pytest.raises(ValueError):
        capi.linear(x, z(64, 88))
    with pytest.raises(ValueError):
        capi.linear(x, w, b=b.to(torch.bfloat16))
    with pytest.raises(ValueError):
        capi.linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        capi.linear_bwd_data(y, w, act="gelu")
    with pytest.raises(ValueError):
        capi.linear_bwd_weight(y, z(5, 96))
    with pytest.raises(capi.SwinWAttnError):
        capi.linear(z(4, 12), z(64, 12))


def test_launches_are_counted():
    x, w, dy = _rand(1, 9000, 64).to(DEV), _rand(2, 96, 64).to(DEV), _rand(3, 9000, 96).to(DEV)
    capi.swin_wattn_launch_count(reset=True)
    capi.linear(x, w)
    assert capi.swin_wattn_launch_count(reset=True) == 1
    capi.linear_bwd_data(dy, w)
    assert capi.swin_wattn_launch_count(reset=True) == 1
    capi.linear_bwd_weight(dy, x)
    assert capi.swin_wattn_launch_count(reset=True) in (1, 2)
    capi.orthogonalize(w)
    assert capi.swin_wattn_launch_count(reset=True) >= 1
    torch.cuda.synchronize()


def test_results_beyond_32_bit_offsets():
    """More than 2^32 bytes of result and of second operand; sampled rows, the last ones among
    them, against fp64."""
    T, K, N = 300_001, 64, 8192
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
    w, b = _rand(2, N, K, std=0.1), _rand(3, N, dtype=torch.float32)
    wd, bd = _dev(w, b)
    y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    pre = torch.empty_like(y)
    st = _status()
    capi.linear(x, wd, bd, act="silu", y=y, pre=pre, status=st)
    _ok(st)
    rows = torch.cat([torch.arange(0, 40), torch.randint(0, T, (200,), generator=torch.Generator().manual_seed(5)),
                      torch.arange(262_100, 262_200), torch.arange(T - 40, T)])
    xr = x[rows.to(DEV)].cpu()
    ry, rz, ty, tz = linear64(xr, w, b, "silu", None)
    assert_within("y", y[rows.to(DEV)], ry, ty)
    assert_within("pre", pre[rows.to(DEV)], rz, tz)
    # the gradient through it: dy is y, the result is written over x's shape
    dx = capi.linear_bwd_data(y, wd, status=st)
    dw, db = capi.linear_bwd_weight(y, x, status=st)
    _ok(st)
    dr, dt = bwd_data64(y[rows.to(DEV)].cpu(), w, None, "none")
    assert_within("dx", dx[rows.to(DEV)], dr, dt)
    cols = torch.tensor([0, 1, 4095, 8191])
    yc = y[:, cols.to(DEV)].double()
    ref = (yc.T @ x.double()).cpu()
    mag = (yc.abs().T @ x.double().abs()).cpu()
    assert_within("dw", dw[cols.to(DEV)], ref, 2000 * 2.0 ** -23 * mag)
    assert_within("db", db[cols.to(DEV)], yc.sum(0).cpu(), 2000 * 2.0 ** -23 * yc.abs().sum(0).cpu())


def test_first_calls_of_a_process_captured():
    """No call before the capture: nothing that the first call of a kernel does may be illegal
    while a stream is captured."""
    import subprocess
    import sys
    code = (
        "import torch\n"
        "from swin_window_attention_gb300 import capi\n"
        "r = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device='cuda')\n"
        "x, xs, w, dy = r(3000, 64), r(5, 64), r(96, 64), r(3000, 96)\n"
        "g = torch.ones(2, 160, 200, device='cuda')\n"
        "torch.cuda.synchronize()\n"
        "graph = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(graph):\n"
        "    o = [capi.linear(x, w), capi.linear(xs, w), capi.linear_bwd_data(dy, w), *capi.linear_bwd_weight(dy, x),\n"
        "         capi.orthogonalize(g), capi.orthogonalize(g[:, :64].contiguous())]\n"
        "graph.replay()\n"
        "torch.cuda.synchronize()\n"
        "assert bool((o[0] == 64).all() and (o[1] == 64).all() and (o[2] == 96).all() and (o[3] == 3000).all())\n"
        "assert bool((o[4] == 3000).all() and torch.isfinite(o[5].float()).all() and torch.isfinite(o[6].float()).all())\n"
        "print('captured')\n")
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stderr[-2000:]


def test_calls_from_several_threads():
    import threading
    x, w, dy = _rand(1, 2500, 64).to(DEV), _rand(2, 96, 64).to(DEV), _rand(3, 2500, 96).to(DEV)
    want = (capi.linear(x, w, act="gelu"), *capi.linear_bwd_weight(dy, x), capi.orthogonalize(w.float()))
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = (capi.linear(x, w, act="gelu"), *capi.linear_bwd_weight(dy, x), capi.orthogonalize(w.float()))
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad
