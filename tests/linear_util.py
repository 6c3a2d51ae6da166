"""Plain fp64 forms of the MLP's products, their gradients and the Newton-Schulz update, and
the error bounds their tests use.

Bounds. A product of two bf16 values is exact in fp32; an fp32 sum of n terms is off by at
most n 2^-23 S, S the sum of the terms' magnitudes (each addition may truncate, so a whole
unit in the last place, not half of one). An activation moves such an error by at most its
largest slope (1.13 for GELU) and adds its own approximation error, ACT_ERR; a derivative is
off by at most SLOPE_ERR (csrc/product.cuh states the fit: the GELU tail to 5e-5 of itself
and 7e-6 in the product; the others to a few fp32 roundings). The result's one rounding to
bf16 is at most 2^-8 of it."""
import numpy as np
import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
ACT_ERR = {"none": 0.0, "relu": 0.0, "gelu": 7.5e-6, "gelu_tanh": 2e-6, "silu": 2e-6}
SLOPE_ERR = {"none": 0.0, "relu": 0.0, "gelu": 3e-5, "gelu_tanh": 4e-6, "silu": 4e-6}
MAX_SLOPE = 1.13
HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24
ADD_F32 = 2.0 ** -23
C_TANH = 0.7978845608028654


def act64(z, act):
    if act == "relu":
        return torch.clamp_min(z, 0.0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 = sigmoid(2 u), which does not cancel in the tail
        return z * torch.sigmoid(2.0 * C_TANH * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if act == "gelu_tanh":
        t = torch.tanh(C_TANH * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C_TANH * (1.0 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s * (1.0 + z * (1.0 - s))


def linear64(x, w, b, act, residual):
    """y, z and the bounds on y and z, in fp64."""
    x, w = x.double(), w.double()
    K = x.shape[-1]
    z, S = x @ w.T, x.abs() @ w.abs().T
    if b is not None:
        z, S = z + b.double(), S + b.double().abs()
    acc = (K + 1) * ADD_F32 * S
    y = act64(z, act)
    tol = MAX_SLOPE * acc + ACT_ERR[act]
    if residual is not None:
        y = y + residual.double()
        tol = tol + HALF_F32 * 2 * y.abs()
    return y, z, tol + HALF_BF16 * (y.abs() + tol), acc + HALF_BF16 * (z.abs() + acc)


def bwd_data64(dy, w, pre, act):
    dy, w = dy.double(), w.double()
    d, S = dy @ w, dy.abs() @ w.abs()
    acc = (w.shape[0] + 1) * ADD_F32 * S
    if act == "none":
        return d, acc + HALF_BF16 * (d.abs() + acc)
    s = slope64(pre.double(), act)
    tol = MAX_SLOPE * acc + (d.abs() + acc) * SLOPE_ERR[act]
    return d * s, tol + HALF_BF16 * ((d * s).abs() + tol)


def bwd_weight64(dy, x, dtype, old_dw=None, old_db=None):
    dy, x = dy.double(), x.double()
    n = dy.shape[0] + 66  # the tokens' additions, and the splits'
    dw, S = dy.T @ x, dy.T.abs() @ x.abs()
    db, Sb = dy.sum(0), dy.abs().sum(0)
    if old_dw is not None:
        dw, S = dw + old_dw.double(), S + old_dw.double().abs()
    if old_db is not None:
        db, Sb = db + old_db.double(), Sb + old_db.double().abs()
    tol = n * ADD_F32 * S
    if dtype == torch.bfloat16:
        tol = tol + HALF_BF16 * (dw.abs() + tol)
    return dw, db, tol, n * ADD_F32 * Sb


def assert_within(name, got, ref, tol):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), name
    excess = (got - ref).abs() - tol - 1e-37
    assert float(excess.max()) <= 0.0, \
        f"{name}: over its bound by {float(excess.max()):.3g} at {int(excess.argmax())}"


# ---- Newton-Schulz -------------------------------------------------------------------

NS = (3.4445, -4.7750, 2.0315)


def orthogonalize64(g, steps, eps=1e-7, scale=1.0, half=False):
    """One matrix in fp64; with half, with every matrix that the kernels hold rounded where and as
    they round it (times 2^8, fp16): X, A about a shift of the diagonal, and the polynomial B, of
    whose diagonal the rounding is taken back from the rows of X. The result then is rounded to
    bf16."""
    a, b, c = NS

    def hold(t):
        return (t * 256.0).to(torch.float16).double() / 256.0 if half else t

    x = g.double()
    x = hold(x / (x.norm() + eps))
    if g.shape[0] > g.shape[1]:
        x = x.T
    eye = torch.eye(x.shape[0], dtype=torch.float64)
    mu = 0.36 / x.shape[0]
    for s in range(steps):
        A = hold(x @ x.T - mu * eye)
        e = a + b * mu + c * mu * mu
        B = e * eye + (b + 2 * c * mu) * A + c * A @ A
        x = (hold(B) @ x) * (B.diagonal() / hold(B).diagonal())[:, None]
        if s < steps - 1:
            x = hold(x)
        mu = 0.75 if mu > 0.12 else mu * e ** 2
    x = scale * (x.T if g.shape[0] > g.shape[1] else x)
    return x.to(torch.bfloat16).double() if half else x
