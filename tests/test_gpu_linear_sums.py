"""How exactly the gradients of a product's weight and bias are summed over many tokens, against
fp64 by the relative 2-norm: a bound per element that has to hold for the worst order of roundings
cannot show a sum that lost a few digits.

The tolerances. A product of 16 tokens brings its 16 terms and the running sum to one exponent and
may cut each of these 17 at its last unit: half a unit lost on average, 0.36 x 2^-23 of the running
sum (a unit is between 2^-24 and 2^-23 of a value, 0.72 x 2^-23 over a binade). A segment of 512 tokens is
32 such products, in which the running sum grows from nothing to the segment's.
* Terms of one sign: every cut has that sign and the running sum is half of the segment's on
  average, 17 x 32 / 2 x 0.36 x 2^-23 = 1.17e-5 of the segment, and so of the whole.
* Terms of random sign: those of the 16 terms cancel, sqrt(16 x 32) x 0.29 units, 0.72 x 2^-23 each, of a
  running sum that is two thirds of the segment's on average (it grows as the square root), 3.8e-7;
  that of the running sum does not, 32 x 2/3 x 0.36 x 2^-23 = 9.2e-7: 1.0e-6 together.
Segments, and the results of splits, are added with rounding to nearest, some 1e-7 more. Where all
of 12544 tokens are one segment, 784 products, it is 24 times as much.

The terms are spread over six decades: sums of bf16 numbers of one size are exact in fp32 for
many thousands of them, and lose nothing wherever they are held."""
import pytest
import torch

from swin_window_attention_gb300 import capi

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {False: 1.2e-6, True: 1.2e-5}  # of terms of one sign?


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _off(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


# tokens, K, N: unsplit on pairs (the sums beside the tile and, of wide ones, in the other
# accumulator), unsplit on single SMs, split
SIZES = [(12544, 1536, 6144), (50176, 1024, 4096), (12544, 1000, 4096), (20001, 512, 8192), (5000, 1536, 6144),
         (700, 1024, 768), (50176, 192, 768), (30011, 48, 104), (520, 96, 64)]


def _spread(g, *shape, one_sign):
    """Numbers spread evenly over the decades from 1e-6 to 1."""
    t = 10.0 ** (-6.0 * torch.rand(*shape, generator=g, device=DEV))
    return (t if one_sign else t * (1 - 2 * torch.randint(0, 2, shape, generator=g, device=DEV))).bfloat16()


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_long_sums(T, K, N, dtype, one_sign):
    """db, which is fp32 beside either type of dw, and dw in fp32; of random terms and of terms of
    one sign, where what is lost at each addition adds up."""
    g = torch.Generator(device=DEV).manual_seed(T + N)
    dy, x = _spread(g, T, N, one_sign=one_sign), _spread(g, T, K, one_sign=one_sign)
    dw, db = torch.empty(N, K, dtype=dtype, device=DEV), torch.empty(N, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    capi.linear_bwd_weight(dy, x, dw=dw, db=db, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert _off(db, dy.double().sum(0)) <= TOL[one_sign]
    if dtype == torch.float32:
        cols = torch.randperm(N, generator=g, device=DEV)[:256]
        assert _off(dw[cols], dy[:, cols].double().T @ x.double()) <= TOL[one_sign]


@pytest.mark.parametrize("T,K,N", [(12544, 1536, 6144), (700, 1024, 768)])
def test_bias_gradient_beside_either_type(T, K, N):
    """Micro-batches added to fp32 sums: db is the same, to the bit, whether dw is fp32 or bf16, as
    both are made of the same segments."""
    g = torch.Generator(device=DEV).manual_seed(N)
    dbs = [torch.zeros(N, device=DEV) for _ in range(2)]
    dws = [torch.zeros(N, K, dtype=t, device=DEV) for t in (torch.float32, torch.bfloat16)]
    ref = torch.zeros(N, dtype=torch.float64, device=DEV)
    for _ in range(3):
        dy = _spread(g, T, N, one_sign=True)
        x = torch.randn(T, K, generator=g, device=DEV).bfloat16()
        for dw, db in zip(dws, dbs):
            capi.linear_bwd_weight(dy, x, dw=dw, db=db, accumulate=True)
        ref += dy.double().sum(0)
    torch.cuda.synchronize()
    assert torch.equal(dbs[0], dbs[1])
    assert _off(dbs[0], ref) <= TOL[True]
