"""Every form of the norms around a block and of their gradients against fp64: each width at which a row changes its shape
(groups of 4 to 32 threads with two to twelve chunks, blocks of 4, 8 and 16 warps with two to four), with a norm before, one
behind and both, for both streams, with more rows than are resident at once."""
import pytest
import torch

from swin_window_attention_gb300 import capi
from tests.test_gpu_block_norm import Case

pytestmark = pytest.mark.gpu

# both ends of each shape's widths, and one between
WIDTHS = [8, 32, 40, 48, 56, 64, 72, 96, 104, 128, 136, 192, 200, 256, 264, 384, 392, 512, 520, 768, 776, 1024, 1032, 1160, 1536,
          1544, 2048, 2056, 2304, 2816, 3080, 4096, 4104, 5000, 6144, 6152, 7168, 7176, 8192]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def tokens(C):
    """Some more rows than the resident blocks of the gradients hold, so that each walks on and some run out earlier."""
    for width, rows in ((48, 20011), (96, 10009), (192, 5003), (384, 2503), (768, 1301), (1536, 701)):
        if C <= width:
            return rows
    return 403


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pre,post", [(1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("C", WIDTHS)
def test_forward_and_backward(C, pre, post, stream):
    T = tokens(C)
    c = Case(T, C, stream=stream, pre=pre, post=post, gate=C % 16 == 0, samples=T if C % 3 else 0, seed=7)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("C", WIDTHS)
def test_rms_without_a_norm_behind(C):
    """As a pre-norm block has it, in few rows and in many."""
    for T in (5, tokens(C)):
        c = Case(T, C, kind="rms", post=False, gate=True, bias=False, alpha=-1.5, seed=9)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("C", [48, 768, 1160, 2304, 7176])
def test_no_norm_at_all(C):
    """The residual sum with gate and depth alone."""
    T = tokens(C)
    c = Case(T, C, pre=False, post=False, samples=T, seed=11)
    c.check_forward()
    c.check_backward()
