"""The fp64 form of the 4-bit formats, which the GPU tests compare with, on known values."""
import torch

from tests.fp4_util import E2M1, E4M3, exact_operand, nearest, quantize64, tensor_scale64


def test_tables():
    assert len(E4M3) == 127 and float(E4M3[-1]) == 448.0 and float(E4M3[8]) == 2.0 ** -6
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(E4M3, want)


def test_ties_go_to_even():
    v = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2, 0.3, 4.9, 5.1, 9.0], dtype=torch.float64)
    assert E2M1[nearest(v, E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4, 0, 0.5, 4, 6, 6]
    h = (E4M3[:-1] + E4M3[1:]) / 2
    want = h.float().to(torch.float8_e4m3fn).double()
    assert torch.equal(E4M3[nearest(h, E4M3)], want)


def test_tensor_scale():
    assert tensor_scale64(torch.tensor([2688.0])) == 1.0 and tensor_scale64(torch.tensor([-2689.0])) == 2.0
    assert tensor_scale64(torch.zeros(3)) == 2.0 ** -90
    assert tensor_scale64(torch.tensor([float("nan"), 1.0, float("inf")])) == tensor_scale64(torch.tensor([1.0]))


def test_exact_operands_are_exact():
    for fmt in ("nvfp4", "mxfp4"):
        x = exact_operand(1, 5, 96, fmt)
        _, byte, values = quantize64(x, fmt, tensor_scale64(x) if fmt == "nvfp4" else None)
        assert torch.equal(values, x.double()) and len(byte.unique()) == 3
