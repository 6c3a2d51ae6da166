"""Failure detection of the MLP's products and the weight update without a GPU fault: the
fault-injection build withholds the completion of the first tile's product (the GEMM site of
include/swin_wattn_debug.h) and shortens the bound of every device wait. Each launch must come
back within seconds with bit 0 of the status word set, and the next call must be right."""
import time

import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.linear_util import assert_within, bwd_weight64, linear64, orthogonalize64

pytestmark = pytest.mark.gpu
DEV = "cuda"
WAIT_NS = 5_000_000
DEFAULT_WAIT_NS = 1_000_000_000


@pytest.fixture(scope="module")
def dbg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build(debug=True)
    lib = capi.load_debug()
    yield lib
    lib.swin_wattn_debug_set_fault(capi.FAULT_NONE, DEFAULT_WAIT_NS)


def _rand(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _armed_then_clean(dbg, call, check):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    try:
        assert dbg.swin_wattn_debug_set_fault(capi.FAULT_GEMM, WAIT_NS) == capi.OK
        t0 = time.monotonic()
        assert call(status.data_ptr()) == capi.OK
        torch.cuda.synchronize()
        elapsed = time.monotonic() - t0
    finally:
        dbg.swin_wattn_debug_set_fault(capi.FAULT_NONE, DEFAULT_WAIT_NS)
    assert int(status.item()) == 1
    assert elapsed < 10.0, f"the timed-out call took {elapsed:.1f} s"
    status.zero_()
    assert call(status.data_ptr()) == capi.OK
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check()


def _stream():
    return torch.cuda.current_stream().cuda_stream


# tokens, K, N: a cluster per tile (few tokens), single SMs, pairs of SMs
@pytest.mark.parametrize("T,K,N", [(20, 1536, 256), (600, 64, 96), (20000, 512, 1024)])
def test_linear_times_out_and_recovers(dbg, T, K, N):
    x, w, b = _rand(1, T, K), _rand(2, N, K, std=K ** -0.5), _rand(3, N, dtype=torch.float32)
    xd, wd, bd = x.to(DEV), w.to(DEV), b.to(DEV)
    y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    rows = torch.randint(0, T, (min(T, 300),), generator=torch.Generator().manual_seed(4))

    def check():
        ref, _, tol, _ = linear64(x[rows], w, b, "gelu", None)
        assert_within("y", y.cpu()[rows], ref, tol)

    _armed_then_clean(dbg, lambda st: dbg.swin_wattn_linear(xd.data_ptr(), wd.data_ptr(), bd.data_ptr(), None,
                                                            y.data_ptr(), None, T, K, N, capi.ACT_GELU, st, _stream()),
                      check)


@pytest.mark.parametrize("T,K,N,dtype", [(3000, 64, 96, torch.float32), (700, 1024, 768, torch.bfloat16)])
def test_weight_gradient_times_out_and_recovers(dbg, T, K, N, dtype):
    dy, x = _rand(1, T, N, std=1e-2), _rand(2, T, K)
    dyd, xd = dy.to(DEV), x.to(DEV)
    dw, db = torch.empty(N, K, dtype=dtype, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(dbg.swin_wattn_linear_bwd_weight_workspace_bytes(T, K, N), dtype=torch.uint8, device=DEV)
    code = capi.FP32 if dtype == torch.float32 else capi.BF16

    def check():
        rw, rb, tw, tb = bwd_weight64(dy, x, dtype)
        assert_within("dw", dw, rw, tw)
        assert_within("db", db, rb, tb)

    _armed_then_clean(dbg, lambda st: dbg.swin_wattn_linear_bwd_weight(dyd.data_ptr(), xd.data_ptr(), dw.data_ptr(),
                                                                       db.data_ptr(), T, K, N, code, 0, ws.data_ptr(),
                                                                       ws.numel(), st, _stream()), check)


# one CTA, a cluster, separate products
@pytest.mark.parametrize("n,r,c", [(2, 96, 200), (1, 64, 1500), (2, 200, 160)])
def test_update_times_out_and_recovers(dbg, n, r, c):
    g = _rand(n + r, n, r, c, dtype=torch.float32)
    gd = g.to(DEV)
    out = torch.empty(n, r, c, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(dbg.swin_wattn_orthogonalize_workspace_bytes(n, r, c), dtype=torch.uint8, device=DEV)

    def check():
        for o, m in zip(out.cpu().double(), g):
            exact, held = orthogonalize64(m, 5), orthogonalize64(m, 5, half=True)
            assert float((o - exact).norm()) <= 1.25 * float((held - exact).norm()) + 1e-4 * float(exact.norm())

    _armed_then_clean(dbg, lambda st: dbg.swin_wattn_orthogonalize(gd.data_ptr(), out.data_ptr(), n, r, c, capi.FP32, 5,
                                                                   1e-7, 1.0, ws.data_ptr(), ws.numel(), st, _stream()),
                      check)
