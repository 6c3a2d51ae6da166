"""The weight update's roundings, as the kernels make them, on the matrices that it meets: the bound
that the header states holds for what they hold, whatever G's rank and spectrum."""
import pytest
import torch

from tests.linear_util import orthogonalize64
from tests.orthogonalize_util import BOUND, held64, matrix


@pytest.mark.parametrize("kind", ["flat", "log", "half", "power0.5", "power1", "power1.5", "power2", "rank1", "rank7",
                                  "rank49"])
@pytest.mark.parametrize("m,n", [(64, 64), (96, 384), (300, 200)])
def test_roundings_stay_within_the_bound(kind, m, n):
    g = matrix(kind, m, n)
    exact = orthogonalize64(g, 5)
    assert float((held64(g, 5) - exact).norm()) <= BOUND * float(exact.norm())
