"""Microscaled 4-bit operands on the GPU: quantisation to the bit against fp64, reading back, special
values, and the product on them: exact on operands whose every result is known to the bit, against fp64
elsewhere; every activation, residuals, streams, replays, bounded waits and the refusals."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.fp4_util import codes_of, exact_operand, quantize64, scale_bytes_of, tensor_scale64
from tests.linear_util import ACT_ERR, ACTS, ADD_F32, HALF_BF16, HALF_F32, MAX_SLOPE, act64, assert_within

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _rand(seed, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def check_quantized(x, fmt, q, ts=None):
    """q against x in 64 bits, to the bit."""
    torch.cuda.synchronize()
    if fmt == "nvfp4" and ts is None:
        ts = tensor_scale64(x)
        assert float(q.tensor_scale) == ts
    code, byte, values = quantize64(x, fmt, ts)
    got, clean = scale_bytes_of(q)
    assert clean
    assert torch.equal(got, byte.reshape(got.shape))
    negative = torch.signbit(x.double()).reshape(code.shape)
    nan = torch.isnan(values)
    have = codes_of(q)
    assert torch.equal(torch.where(nan, 0, have & 7), torch.where(nan, 0, code))
    # the sign of what became zero is the value's, too, where its block's scale is not zero
    live = ~nan & (code > 0)
    assert torch.equal((have >> 3).bool()[live], negative[live])
    return values


SIZES = [(1, 32), (2, 64), (7, 96), (31, 160), (33, 128), (127, 256), (128, 32), (129, 1568), (300, 480), (5, 8192),
         (1000, 1536), (130, 4128)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_to_the_bit_and_read_back(fmt, rows, K, dtype):
    for std in (1.0, 0.02, 300.0):
        x = _rand(rows + K, rows, K, std=std, dtype=dtype)
        x[0, :16] = 0.0
        x[-1] *= torch.exp2(torch.randint(-12, 3, (K // 16,), generator=torch.Generator().manual_seed(K)).float()
                            ).repeat_interleave(16).to(dtype)
        q = capi.quantize_fp4(x.to(DEV), fmt)
        values = check_quantized(x, fmt, q)
        for out in (torch.bfloat16, torch.float32):
            back = capi.dequantize_fp4(q, dtype=out)
            assert back.dtype == out and torch.equal(back.double().cpu(), values)


def test_quantize_ties():
    """Every border between two roundings, and its neighbours, in blocks of every scale mantissa."""
    rows = []
    for m in range(8, 16):
        for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            v = torch.full((16,), t * m / 8, dtype=torch.float32)
            v[1] = torch.nextafter(v[0], torch.tensor(9e9))
            v[2] = torch.nextafter(v[0], torch.tensor(0.0))
            v[3:6] = -v[0:3]
            v[15] = 6.0 * m / 8
            rows += [v, v * 2.0 ** 5]
    x = torch.stack(rows).reshape(-1, 32)
    x[0, 0] = 2688.0 / 2  # the tensor's scale
    check_quantized(x, "nvfp4", capi.quantize_fp4(x.to(DEV), "nvfp4"))
    check_quantized(x, "mxfp4", capi.quantize_fp4(x.to(DEV), "mxfp4"))
    b = x.bfloat16()
    check_quantized(b, "nvfp4", capi.quantize_fp4(b.to(DEV), "nvfp4"))


def test_quantize_with_a_given_scale():
    x = _rand(3, 40, 96, dtype=torch.float32)
    for ts in (2.0 ** -9, 0.5, 2.0 ** -14):  # with the last one every block saturates
        scale = torch.full((1,), ts, device=DEV)
        q = capi.quantize_fp4(x.to(DEV), "nvfp4", scale=scale)
        assert q.tensor_scale.data_ptr() == scale.data_ptr()
        values = check_quantized(x, "nvfp4", q, ts)
        assert torch.equal(capi.dequantize_fp4(q, torch.float32).double().cpu(), values)
    # a result that holds the caller's scale is only written with that scale
    with pytest.raises(ValueError):
        capi.quantize_fp4(x.to(DEV), "nvfp4", out=q)
    assert float(scale) == 2.0 ** -14
    assert capi.quantize_fp4(x.to(DEV), "nvfp4", scale=scale, out=q) is q
    # any positive scale: two roundings more at most
    scale = torch.full((1,), 4.8871 / 2688, device=DEV)
    q = capi.quantize_fp4(x.to(DEV), "nvfp4", scale=scale)
    back = capi.dequantize_fp4(q, torch.float32).double().cpu()
    byte, _ = scale_bytes_of(q)
    top = x.double().reshape(40, -1, 16).abs().amax(-1)
    assert ((back - x.double()).reshape(40, -1, 16).abs().amax(-1) <= top / 6 * 1.13).all()  # half of 2 steps, an E4M3's rounding


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_special_values(fmt):
    x = _rand(5, 6, 128, dtype=torch.float32)
    x[0, 3], x[1, 40], x[2, 127] = float("nan"), float("inf"), float("-inf")
    x[3] = 0.0
    x[4, :32] = -0.0
    x[5, :32] = 3.4e38 if fmt == "mxfp4" else 1e30
    x[5, 32:64] = 1e-44
    values = check_quantized(x, fmt, capi.quantize_fp4(x.to(DEV), fmt))
    back = capi.dequantize_fp4(capi.quantize_fp4(x.to(DEV), fmt), torch.float32).double().cpu()
    assert torch.equal(torch.isnan(back), torch.isnan(values))
    assert torch.isnan(values).sum() == 3 * (16 if fmt == "nvfp4" else 32)
    fine = ~torch.isnan(values) & (values.abs() < 3.4e38)
    assert torch.equal(back[fine], values[fine])


def test_quantize_small_numbers():
    """Subnormal blocks of MXFP4 keep their values; a zero tensor is zero."""
    x = _rand(6, 4, 64, std=1e-38, dtype=torch.float32)
    x[1] *= 1e-3
    values = check_quantized(x, "mxfp4", capi.quantize_fp4(x.to(DEV), "mxfp4"))
    assert (values[0] != 0).any()
    for fmt in FORMATS:
        z = capi.quantize_fp4(torch.zeros(3, 32, device=DEV), fmt)
        assert (capi.dequantize_fp4(z) == 0).all()


def test_no_rows_and_surroundings():
    for fmt in FORMATS:
        e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
        q = capi.quantize_fp4(e, fmt)
        assert capi.dequantize_fp4(q).shape == (0, 64)
        w = capi.quantize_fp4(_rand(1, 24, 64).to(DEV), fmt)
        assert capi.linear_fp4(q, w).shape == (0, 24) and capi.linear_fp4(e, w).shape == (0, 24)
        x = _rand(2, 33, 96).to(DEV)
        ref = capi.quantize_fp4(x, fmt)
        codes = torch.full((35, 48), 9, dtype=torch.uint8, device=DEV)
        room = torch.full((ref.scales.numel() + 64,), 9, dtype=torch.uint8, device=DEV)
        out = capi.Fp4Tensor(codes[1:34], room[32:-32], None if fmt == "mxfp4" else torch.empty(1, device=DEV), capi.FP4_FORMATS[fmt],
                             x.shape)
        assert capi.quantize_fp4(x, fmt, out=out) is out
        torch.cuda.synchronize()
        assert torch.equal(out.codes, ref.codes) and torch.equal(out.scales, ref.scales)
        assert (codes[0] == 9).all() and (codes[34] == 9).all() and (room[:32] == 9).all() and (room[-32:] == 9).all()


# ---- the product ---------------------------------------------------------------------

PRODUCTS = [  # tokens, K, N
    (1, 32, 8), (1, 1536, 1000), (2, 64, 40), (3, 4096, 200), (7, 96, 384), (17, 160, 264), (49, 1536, 512), (64, 64, 64),
    (100, 384, 1152), (127, 288, 32), (128, 256, 256), (129, 224, 1000), (255, 512, 96), (257, 2048, 72), (300, 32, 2000),
    (777, 384, 136), (1000, 192, 768), (4099, 96, 384), (20000, 32, 48), (2100, 512, 2048), (8, 6144, 1536), (1025, 4096, 24),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,N", PRODUCTS)
def test_product_exact(fmt, T, K, N):
    """Operands that 4 bits hold, scales that change from block to block and row to row: every sum is a
    multiple of 1/4 below 2^22, known to the bit, so a scale or an element misplaced, left out or read twice
    shows."""
    x, w = exact_operand(T, T, K, fmt), exact_operand(N + 1, N, K, fmt)
    b = torch.randint(-9, 10, (N,), generator=torch.Generator().manual_seed(3)).float()
    r = torch.randint(-50, 51, (T, N), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    wq = capi.quantize_fp4(w.to(DEV), fmt)
    xq = capi.quantize_fp4(x.to(DEV), fmt)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = capi.linear_fp4(xq, wq, status=st)
    y2 = capi.linear_fp4(x.to(DEV), wq, b.to(DEV), act="relu", residual=r.to(DEV), status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    z = x.double() @ w.double().T
    assert float((x.double().abs() @ w.double().abs().T).max()) < 2 ** 22
    assert torch.equal(y.cpu(), z.to(torch.bfloat16))
    assert torch.equal(y2.cpu(), ((z + b.double()).clamp_min(0) + r.double()).to(torch.bfloat16))


def linear64(xv, wv, b, act, residual):
    """As linear_util.linear64, on decoded operands: products of two 4-bit values and two scales are exact in
    the tensor core's sums; the tensors' scales multiply the sum, two roundings more."""
    K = xv.shape[-1]
    z, S = xv @ wv.T, xv.abs() @ wv.abs().T
    err = (K + 3) * ADD_F32 * S
    if b is not None:
        z = z + b.double()
        err = err + ADD_F32 * (S + b.double().abs())
    y = act64(z, act)
    tol = MAX_SLOPE * err + ACT_ERR[act]
    if residual is not None:
        y = y + residual.double()
        tol = tol + 2 * HALF_F32 * y.abs()
    return y, tol + HALF_BF16 * (y.abs() + tol)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", [(1, 224, 120), (50, 384, 1536), (333, 128, 264), (1500, 96, 104), (5, 1536, 6144)])
def test_product_against_fp64(fmt, act, T, K, N):
    x, w = _rand(T, T, K), _rand(1, N, K, std=2.0 * K ** -0.5)
    b, r = _rand(2, N, dtype=torch.float32), _rand(3, T, N)
    wq = capi.quantize_fp4(w.to(DEV), fmt)
    scale = torch.full((1,), 4.8871 / 2688, device=DEV) if fmt == "nvfp4" else None
    for given in (None, scale):
        xq = capi.quantize_fp4(x.to(DEV), fmt, scale=given)
        xv, wv = (capi.dequantize_fp4(q, torch.float32).double().cpu() for q in (xq, wq))
        for bias, res in ((b, None), (b, r), (None, r), (None, None)):
            y = capi.linear_fp4(x.to(DEV), wq, None if bias is None else b.to(DEV), act=act,
                                residual=None if res is None else r.to(DEV), x_scale=given)
            torch.cuda.synchronize()
            assert_within("y", y, *linear64(xv, wv, bias, act, res))


def test_product_spread_scales():
    """Blocks whose sizes spread over twelve powers of two."""
    for fmt in FORMATS:
        x, w = _rand(1, 200, 512, dtype=torch.float32), _rand(2, 96, 512, dtype=torch.float32)
        up = torch.exp2(torch.randint(-6, 7, (200, 16), generator=torch.Generator().manual_seed(3)).float()).repeat_interleave(32, 1)
        xq, wq = capi.quantize_fp4((x * up).to(DEV), fmt), capi.quantize_fp4((w * up[:96]).to(DEV), fmt)
        y = capi.linear_fp4(xq, wq)
        xv, wv = (capi.dequantize_fp4(q, torch.float32).double().cpu() for q in (xq, wq))
        assert_within("y", y, *linear64(xv, wv, None, "none", None))


@pytest.mark.parametrize("T", [5, 200])
def test_nan_stays_in_its_row(T):
    for fmt in FORMATS:
        x, w = _rand(1, T, 128), _rand(2, 72, 128).to(DEV)
        wq = capi.quantize_fp4(w, fmt)
        ref = capi.linear_fp4(x.to(DEV), wq)
        x[3, 9] = float("nan")
        y = capi.linear_fp4(x.to(DEV), wq)
        keep = torch.arange(T) != 3
        assert torch.equal(y.cpu()[keep], ref.cpu()[keep]) and torch.isnan(y[3]).all()


@pytest.mark.parametrize("T", [3, 300])
def test_residual_in_place_leading_axes_streams_and_replay(T):
    for fmt in FORMATS:
        x, w, r = _rand(1, T, 2, 96).to(DEV), _rand(2, 136, 96).to(DEV), _rand(3, T, 2, 136).to(DEV)
        wq = capi.quantize_fp4(w, fmt)
        want = capi.linear_fp4(x, wq, residual=r)
        assert want.shape == (T, 2, 136)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        other = capi.linear_fp4(x, wq, residual=r, stream=s)
        s.synchronize()
        assert torch.equal(want, other)
        y = r.clone()
        assert capi.linear_fp4(x, wq, residual=y, y=y) is y
        assert torch.equal(want, y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            z = capi.linear_fp4(x, wq, residual=r)
        x.copy_(_rand(7, T, 2, 96))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, capi.linear_fp4(x, wq, residual=r))


def test_surroundings_of_the_result_stay():
    for T, N in ((3, 72), (130, 136), (257, 200)):
        for fmt in FORMATS:
            x, wq = _rand(1, T, 64).to(DEV), capi.quantize_fp4(_rand(2, N, 64).to(DEV), fmt)
            room = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
            capi.linear_fp4(x, wq, y=room[1:-1])
            torch.cuda.synchronize()
            assert (room[0] == 7).all() and (room[-1] == 7).all() and (room[1:-1] != 7).any()


@pytest.mark.parametrize("T,K,N", [(20, 1536, 256), (600, 64, 96), (20000, 512, 1024)])
def test_bounded_waits(T, K, N):
    """The fault-injection build withholds the first tile's completion: the call returns with the status
    word set, and the next one is right."""
    from swin_window_attention_gb300 import build
    build.build(debug=True)
    dbg = capi.load_debug()
    q = [capi.quantize_fp4(_rand(s, n, K).to(DEV), "nvfp4") for s, n in ((1, T), (2, N))]
    want = capi.linear_fp4(*q)
    y = torch.empty_like(want)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call():
        ptrs = [t.data_ptr() for o in q for t in (o.codes, o.scales, o.tensor_scale)]
        assert ptrs == [a for o in q for a in o._at]
        assert dbg.swin_wattn_linear_fp4(*ptrs, None, None, y.data_ptr(), T, K, N, capi.NVFP4, capi.ACT_NONE, status.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream) == capi.OK
        torch.cuda.synchronize()

    try:
        assert dbg.swin_wattn_debug_set_fault(capi.FAULT_GEMM, 5_000_000) == capi.OK
        call()
    finally:
        dbg.swin_wattn_debug_set_fault(capi.FAULT_NONE, 1_000_000_000)
    assert int(status) == 1
    status.zero_()
    call()
    assert int(status) == 0 and torch.equal(y, want)


def test_refusals():
    x, w = _rand(1, 8, 64).to(DEV), _rand(2, 16, 64).to(DEV)
    wq = capi.quantize_fp4(w, "nvfp4")
    with pytest.raises(ValueError):
        capi.quantize_fp4(x, "fp4")
    with pytest.raises(ValueError):
        capi.quantize_fp4(x, "mxfp4", scale=torch.ones(1, device=DEV))
    with pytest.raises(ValueError):
        capi.quantize_fp4(x.half(), "mxfp4")
    with pytest.raises(capi.SwinWAttnError) as e:
        capi.quantize_fp4(_rand(1, 8, 48).to(DEV), "mxfp4")
    assert e.value.status == capi.ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        capi.linear_fp4(capi.quantize_fp4(x, "mxfp4"), wq)
    with pytest.raises(ValueError):
        capi.linear_fp4(capi.quantize_fp4(x, "nvfp4"), wq, x_scale=torch.ones(1, device=DEV))
    with pytest.raises(ValueError):
        capi.linear_fp4(_rand(1, 8, 96).to(DEV), wq)
    with pytest.raises(ValueError):
        capi.linear_fp4(x, wq, torch.ones(15, device=DEV))
    with pytest.raises(capi.SwinWAttnError) as e:
        capi.linear_fp4(x, capi.quantize_fp4(_rand(2, 12, 64).to(DEV), "nvfp4"))
    assert e.value.status == capi.ERR_UNSUPPORTED
    for parts in ((wq.codes, wq.scales[:-512], wq.tensor_scale), (wq.codes, wq.scales, None), (wq.codes[:, ::2], wq.scales,
                  wq.tensor_scale), (wq.codes[:-1], wq.scales, wq.tensor_scale)):
        with pytest.raises(ValueError):
            capi.Fp4Tensor(*parts, "nvfp4", wq.shape)
    with pytest.raises(ValueError):
        capi.Fp4Tensor(wq.codes, wq.scales, wq.tensor_scale, "mxfp4", wq.shape)
    odd = torch.empty(wq.codes.numel() + 1, dtype=torch.uint8, device=DEV)[1:].view_as(wq.codes)
    with pytest.raises(capi.SwinWAttnError) as e:
        capi.linear_fp4(x, capi.Fp4Tensor(odd, wq.scales, wq.tensor_scale, wq.format, wq.shape))
    assert e.value.status == capi.ERR_MISALIGNED
    y = torch.empty(8, 16, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(capi.SwinWAttnError) as e:  # the status word inside the result
        capi.linear_fp4(x, wq, y=y, status=y.view(torch.int32).view(-1)[:1])
    assert e.value.status == capi.ERR_INVALID_ARG
