"""Host-side checks of the MLP's products and the weight update that need no GPU: argument
errors come back before any CUDA call, the workspace sizes, and the Python wrappers' checks."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from swin_window_attention_gb300 import build, capi
    build.build()
    return capi


def test_products_reject_bad_arguments_before_touching_cuda(lib):
    lin = lambda T, K, N, act=0: lib.swin_wattn_linear(*([None] * 6), T, K, N, act, None, None)
    dat = lambda T, K, N, act=0: lib.swin_wattn_linear_bwd_data(*([None] * 4), T, K, N, act, None, None)
    for f in (lin, dat):
        assert f(-1, 64, 64) == lib.ERR_INVALID_ARG
        assert f(4, 64, 64, 5) == lib.ERR_INVALID_ARG and f(4, 64, 64, -1) == lib.ERR_INVALID_ARG
        assert f(4, 60, 64) == lib.ERR_UNSUPPORTED and f(4, 64, 4) == lib.ERR_UNSUPPORTED
        assert f(4, 0, 64) == lib.ERR_UNSUPPORTED and f(4, 64, 32776) == lib.ERR_UNSUPPORTED
        assert f(0, 64, 64) == lib.OK
        assert f(2 ** 31 - 1, 8, 8) == lib.ERR_UNSUPPORTED
        assert f(4, 64, 64) == lib.ERR_INVALID_ARG  # null pointers
    wgt = lambda T, K, N, dt=1, nb=0: lib.swin_wattn_linear_bwd_weight(*([None] * 4), T, K, N, dt, 0, None, nb, None,
                                                                       None)
    assert wgt(-1, 64, 64) == lib.ERR_INVALID_ARG and wgt(4, 64, 64, 2) == lib.ERR_INVALID_ARG
    assert wgt(4, 12, 64) == lib.ERR_UNSUPPORTED and wgt(4, 64, 64) == lib.ERR_INVALID_ARG
    assert wgt(0, 64, 64) == lib.ERR_INVALID_ARG  # no tokens still write dw: null


def test_workspace_sizes(lib):
    f = lib.swin_wattn_linear_bwd_weight_workspace_bytes
    assert f(-1, 64, 64) == 0 and f(4, 60, 64) == 0 and f(4, 64, 0) == 0 and f(2 ** 31 - 1, 8, 8) == 0
    for T, K, N in [(0, 8, 8), (1, 8, 8), (50176, 192, 768), (2 ** 31 - 1024, 8, 8), (12544, 1536, 6144), (1, 32768, 32768)]:
        n = f(T, K, N)
        assert n >= 256 and (n == 256 or n % ((N * K + N) * 4) == 0)
    g = lib.swin_wattn_orthogonalize_workspace_bytes
    assert g(-1, 8, 8) == 0 and g(1, 0, 8) == 0 and g(1, 8, 16385) == 0 and g(65536, 8, 8) == 0
    # two copies of X and two matrices of the smaller side, in 16 bits
    assert g(3, 160, 384) >= 3 * 2 * (2 * 160 * 384 + 2 * 160 * 160) and g(3, 96, 384) >= 256
    assert g(65535, 1024, 1024) >= 65535 * 8 * 1024 * 1024


def test_update_rejects_bad_scalars_before_touching_cuda(lib):
    f = lambda n=1, r=8, c=8, dt=1, steps=5, eps=1e-7, scale=1.0: lib.swin_wattn_orthogonalize(
        None, None, n, r, c, dt, steps, eps, scale, None, 0, None, None)
    bad = lib.ERR_INVALID_ARG
    assert f(n=-1) == bad and f(dt=7) == bad and f(steps=0) == bad and f(steps=21) == bad
    assert f(eps=0.0) == bad and f(eps=-1.0) == bad and f(eps=np.inf) == bad and f(scale=np.nan) == bad
    assert f(r=0) == lib.ERR_UNSUPPORTED and f(c=20000) == lib.ERR_UNSUPPORTED and f(n=70000) == lib.ERR_UNSUPPORTED
    assert f(n=0) == lib.OK and f() == bad


def test_update_rejects_a_subnormal_eps(lib):
    f = lambda eps: lib.swin_wattn_orthogonalize(None, None, 0, 8, 8, 1, 5, eps, 1.0, None, 0, None, None)
    assert f(1e-40) == lib.ERR_INVALID_ARG and f(2.0 ** -149) == lib.ERR_INVALID_ARG and f(2.0 ** -126) == lib.OK


def test_update_rejects_a_tiny_scale(lib):
    f = lambda scale: lib.swin_wattn_orthogonalize(None, None, 0, 8, 8, 1, 5, 1e-7, scale, None, 0, None, None)
    assert f(1e-38) == lib.ERR_INVALID_ARG and f(-(2.0 ** -101)) == lib.ERR_INVALID_ARG
    assert f(0.0) == lib.OK and f(-(2.0 ** -100)) == lib.OK and f(1e38) == lib.OK


def test_wrappers_refuse_host_tensors(lib):
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.bfloat16)
    for call in (lambda: lib.linear(x, w), lambda: lib.linear_bwd_data(x, w), lambda: lib.linear_bwd_weight(x, x),
                 lambda: lib.orthogonalize(w)):
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
    """2^32 + 8 of anything would arrive as 8."""
    n = 2 ** 32 + 8
    x, w = _Described(n, 8), _Described(8, 8)
    for call in (lambda: lib.linear(x, w), lambda: lib.linear(_Described(n // 8, 8, 8), w),
                 lambda: lib.linear(_Described(4, 8), _Described(n, 8)),
                 lambda: lib.linear_bwd_data(x, w), lambda: lib.linear_bwd_data(_Described(4, 8), _Described(8, n)),
                 lambda: lib.linear_bwd_weight(x, x), lambda: lib.orthogonalize(_Described(n, 1, 1)),
                 lambda: lib.orthogonalize(_Described(8, 8), steps=n)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_update_keeps_singular_values_in_its_band():
    """The iteration itself (the plain form the GPU tests compare with): singular values of
    any positive size end in [0.65, 1.25], and the fp16 roundings change the result by less
    than 2^-8 of its norm on a random matrix."""
    from tests.linear_util import orthogonalize64
    g = torch.randn(64, 100, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    s = torch.linalg.svdvals(orthogonalize64(g, 5))
    assert float(s.min()) > 0.65 and float(s.max()) < 1.25
    e, h = orthogonalize64(g, 5), orthogonalize64(g, 5, half=True)
    assert float((h - e).norm() / e.norm()) < 2.0 ** -8
