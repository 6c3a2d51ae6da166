"""Plain fp64 forms of the residual sum with its norms and of its gradients, with the error
bounds their tests use.

Bounds, with u = 2^-24, the largest relative error of an fp32 rounding. A sum over a row is made of
at most 24 additions in a thread, five of a warp's and sixteen of a block's, so it is off by at most
N u S, N = 64 and S the sum of the terms' magnitudes. With s = sqrt(var + eps) (the norm's divisor) and
inputs off by at most e a row:
* d = v - mean is off by E = 2 e + N u mean|v| + u |d|;
* the reciprocal of s, relatively, by R = (E + e) / s + N u + 2^-21 (the hardware's reciprocal square
  root is off by 2^-22, the mean of squares by N u and by 2 E |d|, at most 2 E s s);
* vhat = d / s by E / s + (|vhat| + E / s) R, and vhat w + b by |w| times that and two roundings.
The gradient through a norm, r (g - mean g - vhat mean(g vhat)), for g off by eg and vhat off by ev:
the means are off by N u mean|g| + eg and N u mean|g vhat| + eg mean|vhat| + ev mean|g|.
Sums over T tokens are off by (T + N) u times the magnitudes and by what their terms are off.
A result's one rounding to bf16 is at most 2^-8 of it (half a step is 2^-9 of the power of two above)."""
import torch

U = 2.0 ** -24
N = 64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def normalise64(v, kind, eps, err=0.0):
    """vhat, 1 / s and the bound on vhat, for v off by at most err (a number or a column)."""
    d = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    s = (d.square().mean(-1, keepdim=True) + eps).sqrt()
    E = 2 * err + (N * U * v.abs().mean(-1, keepdim=True) if kind == "layer" else 0.0) + U * d.abs()
    top = E.amax(-1, keepdim=True)
    vhat = d / s
    R = (top + err) / s + N * U + 2.0 ** -21
    return vhat, 1 / s, E / s + (vhat.abs() + top / s) * R, R


def affine64(vhat, ev, wb):
    w, b = wb[0].double(), None if wb[1] is None else wb[1].double()
    out = vhat * w if b is None else vhat * w + b
    mag = vhat.abs() * w.abs() + (0 if b is None else b.abs())
    return out, ev * w.abs() + 2 * U * mag


def of_tokens(keep, T):
    return keep.double().repeat_interleave(T // keep.numel())[:, None]


def forward64(x, f, pre, post, gate, keep, alpha, kind, eps, stream):
    """(y, tolerance) and (h, tolerance), either None."""
    y, ey = x.double(), torch.zeros_like(x, dtype=torch.float64)
    first = None
    if f is not None:
        u, eu = f.double(), torch.zeros_like(y)
        if post is not None:
            vhat, _, ev, _ = normalise64(u, kind, eps)
            u, eu = affine64(vhat, ev, post)
        if gate is not None:
            u, eu = u * gate.double(), (eu + U * u.abs()) * gate.double().abs()
        if keep is not None:
            k = of_tokens(keep, x.shape[0])
            u, eu = u * k, (eu + U * u.abs()) * k.abs()
        mag = (alpha * y).abs() + u.abs()
        y, ey = alpha * y + u, eu + 3 * U * mag
        first = (y, ey + HALF[stream] * (y.abs() + ey))
    second = None
    if pre is not None:
        vhat, _, ev, _ = normalise64(y, kind, eps, ey.amax(-1, keepdim=True))
        h, eh = affine64(vhat, ev, pre)
        second = (h, eh + HALF[torch.bfloat16] * (h.abs() + eh))
    return first, second


def through64(g, eg, vhat, ev, r, R, kind):
    m1 = (g * vhat).mean(-1, keepdim=True)
    e1 = N * U * (g * vhat).abs().mean(-1, keepdim=True) + (eg * vhat.abs() + ev * g.abs()).mean(-1, keepdim=True)
    m0 = g.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(m1)
    e0 = N * U * g.abs().mean(-1, keepdim=True) + eg.mean(-1, keepdim=True) if kind == "layer" else 0.0
    inner = g - m0 - vhat * m1
    mag = g.abs() + m0.abs() + (vhat * m1).abs()
    ei = eg + e0 + ev * m1.abs() + (vhat.abs() + ev) * e1 + 3 * U * mag
    return r * inner, r * (ei + (inner.abs() + ei) * (R + U))


def backward64(y, f, dh, dy, pre, post, gate, keep, alpha, kind, eps, stream):
    """{name: (value, tolerance)} for dx, df and the parameters' gradients."""
    y, T, out = y.double(), y.shape[0], {}
    zero = torch.zeros_like(y)

    def total(terms, err):
        return terms.sum(0), (T + N) * U * terms.abs().sum(0) + err.sum(0)

    d, ed = (zero if dy is None else dy.double()), zero
    if pre is not None:
        dh = dh.double()
        vhat, r, ev, R = normalise64(y, kind, eps)
        out["pre_weight"] = total(dh * vhat, dh.abs() * (ev + U * vhat.abs()))
        if pre[1] is not None:
            out["pre_bias"] = total(dh, zero)
        g = dh * pre[0].double()
        t, et = through64(g, U * g.abs(), vhat, ev, r, R, kind)
        d, ed = d + t, et + U * (d.abs() + t.abs())
    out["dx"] = (alpha * d, abs(alpha) * ed + U * (alpha * d).abs() + HALF[stream] * ((alpha * d).abs() + abs(alpha) * ed))
    if f is None:
        return out
    if keep is not None:
        k = of_tokens(keep, T)
        d, ed = d * k, (ed + U * d.abs()) * k.abs()
    u, eu = f.double(), zero
    if post is not None:
        fhat, r, ef, R = normalise64(u, kind, eps)
        P, eP = total(d * fhat, ed * fhat.abs() + d.abs() * (ef + U * fhat.abs()))
        Q, eQ = total(d, ed)
        gt = torch.ones(y.shape[1], dtype=torch.float64) if gate is None else gate.double()
        out["post_weight"] = (gt * P, gt.abs() * eP + U * (gt * P).abs())
        if post[1] is not None:
            out["post_bias"] = (gt * Q, gt.abs() * eQ + U * (gt * Q).abs())
        if gate is not None:
            w, b = post[0].double(), torch.zeros_like(P) if post[1] is None else post[1].double()
            out["gate"] = (w * P + b * Q, w.abs() * eP + b.abs() * eQ + 2 * U * ((w * P).abs() + (b * Q).abs()))
        g = d * gt * post[0].double()
        d, ed = through64(g, (ed + 2 * U * d.abs()) * (gt * post[0].double()).abs(), fhat, ef, r, R, kind)
    else:
        if gate is not None:
            out["gate"] = total(d * u, ed * u.abs() + U * (d * u).abs())
            d, ed = d * gate.double(), (ed + U * d.abs()) * gate.double().abs()
    out["df"] = (d, ed + HALF[torch.bfloat16] * (d.abs() + ed))
    return out


def assert_close(name, got, want):
    ref, tol = want
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), name
    excess = (got - ref).abs() - tol - 1e-37
    assert float(excess.max()) <= 0.0, f"{name}: over its bound by {float(excess.max()):.3g} at {int(excess.argmax())}"
