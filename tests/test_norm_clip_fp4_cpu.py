"""Host-side checks of the norms, the clipping and the 4-bit operands that need no GPU: argument errors
come back before any CUDA call, sizes of workspaces and scales, and the Python wrappers' checks."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from swin_window_attention_gb300 import build, capi
    build.build()
    return capi


def test_norms_reject_bad_arguments_before_touching_cuda(lib):
    bad, un, ok = lib.ERR_INVALID_ARG, lib.ERR_UNSUPPORTED, lib.OK
    # pointers that are never read: the checks come before
    x, f, w, g, k, y, h = (1 << 12) + 4096, 1 << 14, 1 << 15, 1 << 16, 1 << 17, 1 << 18, 1 << 19

    def fwd(T=4, C=64, x=x, f=f, pw=w, pb=None, qw=None, qb=None, gate=None, keep=None, y=y, h=h, samples=1, dtype=0, kind=0,
            alpha=1.0, eps=1e-5):
        return lib.swin_wattn_block_norm(x, f, pw, pb, qw, qb, gate, keep, y, h, T, C, samples, dtype, kind, alpha, eps, None)

    assert fwd(T=-1) == bad and fwd(dtype=2) == bad and fwd(kind=2) == bad and fwd(kind=-1) == bad
    assert fwd(eps=0.0) == bad and fwd(eps=float("nan")) == bad and fwd(eps=1e-40) == bad and fwd(eps=float("inf")) == bad
    assert fwd(alpha=float("inf")) == bad
    assert fwd(C=0) == un and fwd(C=60) == un and fwd(C=8200) == un and fwd(T=2 ** 31 - 1) == un
    assert fwd(keep=k, samples=0) == bad and fwd(keep=k, samples=3) == bad
    assert fwd(T=0) == ok and fwd(T=0, x=None, f=None, y=None, h=None, pw=None) == ok
    assert fwd(f=None) == bad and fwd(f=None, y=None, gate=g) == bad and fwd(f=None, y=None, qw=w) == bad
    assert fwd(f=None, y=None, pw=None, h=None) == bad and fwd(y=None) == bad and fwd(h=None) == bad and fwd(x=None) == bad
    assert fwd(pw=None) == bad and fwd(pw=None, h=None, pb=w) == bad and fwd(qb=w) == bad

    def bwd(T=4, C=64, f=f, dh=h, dy=None, pw=w, qw=None, qb=None, gate=None, keep=None, dx=y, df=g, grads=(None,) * 5, ws=k,
            nb=1 << 20, samples=1, eps=1e-5):
        return lib.swin_wattn_block_norm_bwd(x, f, dh, dy, pw, qw, qb, gate, keep, dx, df, *grads, T, C, samples, 0, 0, 1.0, eps,
                                             0, ws, nb, None)

    assert bwd(T=-1) == bad and bwd(eps=0.0) == bad and bwd(C=12) == un and bwd(keep=k, samples=3) == bad
    assert bwd(dh=None) == bad and bwd(pw=None) == bad and bwd(dh=None, pw=None) == bad and bwd(df=None) == bad
    assert bwd(f=None) == bad and bwd(dx=None) == bad and bwd(ws=None) == bad and bwd(nb=16) == bad
    assert bwd(grads=(None, None, w, None, None)) == bad and bwd(grads=(None, None, None, None, w)) == bad
    assert bwd(pw=None, dh=None, dy=h, grads=(w, None, None, None, None)) == bad
    assert bwd(f=None, df=None, gate=g) == bad
    assert bwd(T=0) == ok and bwd(T=0, f=None, dh=None, dx=None, df=None, ws=None) == ok


def test_sizes(lib):
    f = lib.swin_wattn_block_norm_bwd_workspace_bytes
    assert f(-1, 64) == 0 and f(4, 60) == 0 and f(4, 8200) == 0 and f(2 ** 31 - 1, 8) == 0
    for T in (0, 1, 33, 10 ** 6, 2 ** 31 - 1024):
        for C in range(8, 8193, 8):
            n = f(T, C)
            assert 256 <= n <= 152 * 18 * 4 * C * 4 + 256
            assert T == 0 or n % (16 * C) == 0 or n == 256
    s = lib.swin_wattn_fp4_scale_bytes
    assert s(-1, 32, 0) == 0 and s(4, 48, 0) == 0 and s(4, 32, 2) == 0 and s(4, 32800, 0) == 0
    assert s(0, 32, 0) == 0 and s(1, 32, 0) == 512 and s(128, 64, 0) == 512 and s(129, 96, 0) == 2048
    assert s(1, 128, 1) == 512 and s(1, 160, 1) == 1024
    assert s(2 ** 31 - 1024, 32768, 0) == (2 ** 31 - 1024) // 128 * 512 * 512
    from swin_window_attention_gb300.capi import _fp4_sizes
    for rows, K in ((0, 32), (1, 32), (127, 4128), (129, 96), (1000, 32768)):
        for fmt in (0, 1):
            assert _fp4_sizes(torch.Size((rows, K)), fmt) == (rows, K, s(rows, K, fmt))
    w = lib.swin_wattn_linear_fp4_workspace_bytes
    assert w(-1, 32, 8, 0, 0) == 0 and w(1, 40, 8, 0, 0) == 0 and w(1, 32, 8, 5, 0) == 0 and w(1, 32, 9, 0, 0) == 0
    assert w(7, 96, 8, 0, 0) >= 7 * 48 + s(7, 96, 0) + 4 + lib.swin_wattn_fp4_workspace_bytes()
    assert w(1, 6144, 1536, 0, 1) == 0 and w(1, 6144, 1536, 1, 0) == 0  # quantised by the product
    assert w(300, 96, 8, 0, 1) > 0 and w(300, 96, 8, 1, 0) > 0


def test_fp4_rejects_bad_arguments_before_touching_cuda(lib):
    bad, un, ok = lib.ERR_INVALID_ARG, lib.ERR_UNSUPPORTED, lib.OK
    p = 1 << 14

    def q(rows=4, K=64, fmt=0, dtype=0, given=0, x=p, c=p, s=p, ts=p, ws=p, nb=1 << 20):
        return lib.swin_wattn_fp4_quantize(x, c, s, ts, rows, K, fmt, dtype, given, ws, nb, None)

    assert q(rows=-1) == bad and q(fmt=2) == bad and q(dtype=5) == bad and q(K=48) == un and q(K=0) == un
    assert q(ts=None) == bad and q(fmt=1) == bad and q(ws=None) == bad and q(nb=4) == bad and q(x=None) == bad
    assert q(rows=0, given=1) == ok and q(rows=0, fmt=1, ts=None, ws=None) == ok

    def d(rows=4, K=64, fmt=0, dtype=0, c=p, s=p, ts=p, o=p):
        return lib.swin_wattn_fp4_dequantize(c, s, ts, o, rows, K, fmt, dtype, None)

    assert d(rows=-1) == bad and d(ts=None) == bad and d(fmt=1) == bad and d(K=40) == un and d(o=None) == bad and d(rows=0) == ok

    def lin(T=4, K=64, N=64, fmt=0, act=0, xs=p, ws=p, y=p, xc=p):
        return lib.swin_wattn_linear_fp4(xc, p, xs, p, p, ws, None, None, y, T, K, N, fmt, act, None, None)

    assert lin(T=-1) == bad and lin(act=5) == bad and lin(fmt=3) == bad and lin(xs=None) == bad and lin(fmt=1) == bad
    assert lin(K=40) == un and lin(N=12) == un and lin(T=2 ** 31 - 1) == un and lin(y=None) == bad and lin(xc=None) == bad
    assert lin(T=0) == ok

    def of(T=4, K=64, N=64, fmt=0, dtype=0, act=0, xs=p, wt=p, x=p, ws=p, nb=1 << 20):
        return lib.swin_wattn_linear_fp4_of(x, xs, p, p, wt, None, None, p, T, K, N, fmt, dtype, act, ws, nb, None, None)

    assert of(T=-1) == bad and of(dtype=2) == bad and of(fmt=1, wt=None) == bad and of(fmt=1, xs=None) == bad and of(K=40) == un
    assert of(x=None) == bad and of(ws=None) == bad and of(nb=8) == bad and of(T=0) == ok


def test_clip_plan_rejects_bad_arguments(lib):
    plan = lib.swin_wattn_clip_plan
    for grads, outs, sizes, dtypes in (([1 << 14], [1 << 14], [-1], [1]), ([1 << 14], [1 << 14], [4], [3]), ([None], [1 << 14], [4], [1]),
                                       ([1 << 14], [None], [4], [1]), ([1 << 14], [1 << 14], [2 ** 41], [1])):
        rc, h = plan(grads, outs, sizes, dtypes, 1 << 16, 1 << 20, None)
        assert rc == lib.ERR_INVALID_ARG and h is None
    for ptr, size in ((None, 1 << 20), (1 << 16, 16)):
        rc, h = plan([1 << 14], [1 << 14], [4], [1], ptr, size, None)
        assert rc == lib.ERR_INVALID_ARG and h is None
    lb = lib.swin_wattn_clip_list_bytes
    assert lb([-1], [1]) == 0 and lb([4], [7]) == 0 and lb([], []) == 256 and lb([0, 0], [0, 1]) == 256
    assert lb([2048 * 9], [0]) == 32 * 9 and lb([2048 * 9 + 1] * 100, [0] * 100) == 32 * 1000
    assert lb([2 ** 38], [1]) <= 2 << 20
    assert lib.swin_wattn_clip_grad_norm(None, 1.0, 1.0, 0.0, None, 1 << 14, 1 << 20, None) == lib.ERR_BAD_PLAN
    assert lib.swin_wattn_clip_grad_norm(1 << 14, 1.0, 1.0, 0.0, None, 1 << 14, 1 << 20, None) == lib.ERR_BAD_PLAN
    assert lib.swin_wattn_clip_workspace_bytes() > 0 and lib.swin_wattn_clip_destroy(None) == lib.OK
    assert lib.swin_wattn_clip_destroy(1 << 14) == lib.ERR_BAD_PLAN


def test_wrappers_refuse_host_tensors(lib):
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.ones(32)
    for call in (lambda: lib.block_norm(x, pre=(w, w)), lambda: lib.block_norm_bwd(x, dh=x, pre=(w, w)), lambda: lib.GradClip([w]),
                 lambda: lib.quantize_fp4(x), lambda: lib.Fp4Tensor(x.view(torch.uint8), x.view(torch.uint8), None, "mxfp4", (4, 32))):
        with pytest.raises(ValueError):
            call()


class _Described:
    """What the wrappers ask a tensor about, for sizes that no test allocates."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, "cuda:0"

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def test_wrappers_refuse_sizes_that_no_int_holds(lib):
    n = 2 ** 32 + 8
    for call in (lambda: lib.block_norm(_Described(n, 8), pre=(None, None)), lambda: lib.block_norm(_Described(8, n), pre=(None, None)),
                 lambda: lib.block_norm_bwd(_Described(n, 8), dh=_Described(n, 8), pre=(None, None)),
                 lambda: lib.quantize_fp4(_Described(n, 32)), lambda: lib.quantize_fp4(_Described(8, n, 32)),
                 lambda: lib.Fp4Tensor(_Described(n, 16), None, None, "mxfp4", (n, 32))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
