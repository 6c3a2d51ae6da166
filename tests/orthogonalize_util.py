"""Matrices that a weight update meets beside broad ones, and the Newton-Schulz iteration in fp64
with the roundings of the kernels.

A raw gradient's rank is at most its number of tokens, and a momentum's singular values fall off:
the exact iteration leaves the directions that G does not have empty, while noise in them grows
by 3.44 a step.

What the kernels hold: A and B = a I + b A + c A^2 in fp16 times 2^8 (A less a shift of its diagonal;
of B's diagonal the rounding is taken back from the rows of X), X in two fp16 parts times 2^14,
its rounding and what that leaves; A is made of the larger part. Over spectra from flat to
k^-2, halves a thousandfold apart and ranks from 1, five steps of that end within 2e-3 (relative
2-norm) of the exact result with a smaller side of at least 64 (1.75e-3 was the largest of them)."""
import torch

from tests.linear_util import HALF_BF16, NS

BOUND = 2e-3  # of the result before its rounding to bf16: five steps, smaller side >= 64


def orthogonal_factors(m, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    u, _ = torch.linalg.qr(torch.randn(m, k, generator=g, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(n, k, generator=g, dtype=torch.float64))
    return u, v


def matrix(kind, m, n, seed=0):
    """One fp32 matrix: "rank<r>", a product of r tokens' gradients and inputs; "power<p>",
    singular values k^-p; "log", 1 to 0.01; "half", half of them 1 and half 0.01; "flat"."""
    k = min(m, n)
    if kind.startswith("rank"):
        r, g = int(kind[4:]), torch.Generator().manual_seed(seed)
        return 1e-3 * (torch.randn(m, r, generator=g, dtype=torch.float64)
                       @ torch.randn(r, n, generator=g, dtype=torch.float64)).float()
    i = torch.arange(1, k + 1, dtype=torch.float64)
    s = {"log": torch.logspace(0, -2, k, dtype=torch.float64), "half": torch.where(2 * i <= k, 1.0, 0.01).double(),
         "flat": torch.ones(k, dtype=torch.float64)}.get(kind)
    if s is None:
        s = i ** -float(kind[5:])
    u, v = orthogonal_factors(m, n, k, seed)
    return ((u * s) @ v.T).float()


def held64(g, steps, eps=1e-7, scale=1.0):
    """The result before its rounding to bf16, with what the kernels hold rounded as they round it."""
    a, b, c = NS

    def hold(t):
        return (t * 256.0).to(torch.float16).double() / 256.0

    def part(t):
        return (t * 16384.0).to(torch.float16).double() / 16384.0

    x = g.double()
    x = x / (x.norm() + eps)
    if g.shape[0] > g.shape[1]:
        x = x.T
    eye = torch.eye(x.shape[0], dtype=torch.float64)
    mu = 0.36 / x.shape[0]
    for _ in range(steps):
        high = part(x)
        low = part(x - high)
        A = hold(high @ high.T - mu * eye)
        e = a + b * mu + c * mu * mu
        B = e * eye + (b + 2 * c * mu) * A + c * A @ A
        x = (hold(B) @ (high + low)) * (B.diagonal() / hold(B).diagonal())[:, None]
        mu = 0.75 if mu > 0.12 else mu * e ** 2
    return scale * (x.T if g.shape[0] > g.shape[1] else x)


def assert_update(out, g, exact, steps, bound=BOUND, model=True):
    """`out` in bf16 of the exact result: within `bound` and one rounding, and, with `model`, within a
    quarter above the error that the held matrices' roundings leave (room for roundings that fall the
    other way, of which matrices of a few entries have too few to average)."""
    size, err = float(exact.norm()), float((out - exact).norm())
    # |bf16(x) - exact| <= |x - exact| + 2^-8 |x|, |x| <= (1 + bound) |exact|
    assert err <= (bound + HALF_BF16 * (1.0 + bound)) * size, (err / size, bound)
    if model:
        held = float((held64(g, steps).to(torch.bfloat16).double() - exact).norm())
        assert err <= 1.25 * held + 1e-4 * size, (err / size, held / size)
