"""The operators of a block's dense half that are measured, with their plain forms.

A Swin block is the attention sub-block and an MLP; training it needs the products' own
gradients and an update of the weights. Four operators cover that:

* ``linear``: y = residual + act(x W^T + b), optionally keeping the pre-activation;
* ``linear_bwd_data``: dx = (dy W) * act'(pre), the gradient of a product's input, taken
  through the activation that made that input;
* ``linear_bwd_weight``: dW = dy^T x and db = column sums of dy;
* ``orthogonalize``: a stack of weight updates brought near orthogonal by Newton-Schulz
  products.

``run`` computes them in elementary torch operations in fp32, or, where ``own`` is set,
through the package's entry points; ``exact`` in fp64.
"""
import math

import torch

own = False

_DEV = "cuda"
_NS = (3.4445, -4.7750, 2.0315)  # coefficients of the odd quintic of one Newton-Schulz step
_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases -----------------------------------------------------------------------------

def _linear(T, K, N, act="none", bias=True, residual=False, pre=False):
    return {"op": "linear", "tokens": T, "K": K, "N": N, "act": act, "bias": bias, "residual": residual, "pre": pre}


def _bwd_data(T, K, N, act="none"):
    return {"op": "linear_bwd_data", "tokens": T, "K": K, "N": N, "act": act}


def _bwd_weight(T, K, N, out="fp32", bias=True):
    return {"op": "linear_bwd_weight", "tokens": T, "K": K, "N": N, "out": out, "bias": bias}


def _orth(count, rows, cols, dtype="fp32", steps=5):
    return {"op": "orthogonalize", "count": count, "rows": rows, "cols": cols, "dtype": dtype, "steps": steps}


def listed():
    return [
        # the classifier head on one pooled token: serving one image, latency counts
        dict(_linear(1, 1536, 1000), name="head_one_token"),
        # the MLP's first product on the last stage of one 224 image (one 7 x 7 window)
        dict(_linear(49, 1536, 6144, act="gelu"), name="fc1_one_window"),
        # the first product in training at the first stage, 16 images of 56 x 56 tokens: the
        # pre-activation is kept for the backward
        dict(_linear(50176, 192, 768, act="gelu", pre=True), name="fc1_stage1_train"),
        # the second product with the shortcut, a ragged number of tokens
        dict(_linear(12561, 6144, 1536, residual=True), name="fc2_residual_ragged"),
        # gradient of a small qkv projection's input, an odd number of tokens
        dict(_bwd_data(777, 384, 1152), name="dgrad_qkv_small"),
        # gradient through the second product and the GELU at the third stage, 64 images
        dict(_bwd_data(12544, 2048, 512, act="gelu"), name="dgrad_fc2_gelu"),
        # weight gradient of a few ragged tokens
        dict(_bwd_weight(100, 384, 1152), name="wgrad_few_tokens"),
        # weight gradient at the first stage: a long contraction, a small result
        dict(_bwd_weight(50176, 192, 768), name="wgrad_stage1_long"),
        # weight gradient of the last stage's wide product, rounded to bf16 for a bf16 optimiser
        dict(_bwd_weight(12544, 1536, 6144, out="bf16"), name="wgrad_wide_bf16"),
        # the update of one small projection
        dict(_orth(1, 96, 384), name="orth_one_small"),
        # the updates of eight tall first products at the third stage, kept in bf16
        dict(_orth(8, 2048, 512, dtype="bf16"), name="orth_stack_tall"),
        # the updates of two wide products of the last stage
        dict(_orth(2, 1536, 6144), name="orth_wide"),
    ]


_MAX_FLOPS = 2.3e11       # of a drawn product
_MAX_ELEMENTS = 1.2e8     # of a drawn product's operands and results


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo=32, hi=6144):
    return max(lo // 8, _log(rng, lo, hi) // 8) * 8


def draw(rng):
    op = rng.choice(("linear", "linear_bwd_data", "linear_bwd_weight", "orthogonalize"))
    if op == "orthogonalize":
        m, n = _log(rng, 24, 1536), _log(rng, 64, 6144)
        rows, cols = (m, n) if rng.random() < 0.5 else (n, m)
        count = _log(rng, 1, 16)
        lo, hi = min(m, n), max(m, n)
        while count > 1 and count * (3.0 * lo * lo * hi + lo ** 3) > 9.0e10:
            count -= 1
        return _orth(count, rows, cols, rng.choice(("bf16", "fp32")), rng.choice((3, 5, 5, 6)))
    T, K, N = _log(rng, 1, 50176), _width(rng), _width(rng)
    T = max(1, int(min(T, _MAX_FLOPS / (2.0 * K * N), _MAX_ELEMENTS / (K + 2.0 * N))))
    act = rng.choice(_ACTS)
    if op == "linear":
        return _linear(T, K, N, act, rng.random() < 0.8, rng.random() < 0.4, rng.random() < 0.4)
    if op == "linear_bwd_data":
        return _bwd_data(T, K, N, act)
    return _bwd_weight(T, K, N, rng.choice(("fp32", "bf16")), rng.random() < 0.8)


# ---- inputs ----------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=_DEV, dtype=torch.float32) * std).to(dtype)

    st = {"case": case}
    if case["op"] == "orthogonalize":
        n, r, c = case["count"], case["rows"], case["cols"]
        # a momentum buffer: a few strong directions over a broad remainder, values of a gradient
        k = min(8, r, c)
        strong = normal(n, r, k, dtype=torch.float32) @ normal(n, k, c, dtype=torch.float32)
        st["g"] = ((strong * 0.5 + normal(n, r, c, dtype=torch.float32)) * 1e-3).to(_DT[case["dtype"]])
        st["out"] = torch.empty(n, r, c, dtype=torch.bfloat16, device=_DEV)
        if own:
            from swin_window_attention_gb300 import capi
            st["workspace"] = torch.empty(capi.swin_wattn_orthogonalize_workspace_bytes(n, r, c), dtype=torch.uint8,
                                          device=_DEV)
        return st
    T, K, N = case["tokens"], case["K"], case["N"]
    if case["op"] == "linear":
        st["x"] = normal(T, K)
        st["w"] = normal(N, K, std=K ** -0.5)
        st["b"] = normal(N, std=0.1, dtype=torch.float32) if case["bias"] else None
        st["residual"] = normal(T, N) if case["residual"] else None
        st["y"] = torch.empty(T, N, dtype=torch.bfloat16, device=_DEV)
        st["pre"] = torch.empty(T, N, dtype=torch.bfloat16, device=_DEV) if case["pre"] else None
    elif case["op"] == "linear_bwd_data":
        st["dy"] = normal(T, N, std=1e-3)
        st["w"] = normal(N, K, std=K ** -0.5)
        st["pre"] = normal(T, K) if case["act"] != "none" else None
        st["dx"] = torch.empty(T, K, dtype=torch.bfloat16, device=_DEV)
    else:
        st["dy"] = normal(T, N, std=1e-3)
        st["x"] = normal(T, K)
        st["dw"] = torch.empty(N, K, dtype=_DT[case["out"]], device=_DEV)
        st["db"] = torch.empty(N, dtype=torch.float32, device=_DEV) if case["bias"] else None
        if own:
            from swin_window_attention_gb300 import capi
            st["workspace"] = torch.empty(capi.swin_wattn_linear_bwd_weight_workspace_bytes(T, K, N),
                                          dtype=torch.uint8, device=_DEV)
    return st


# ---- one pass --------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from swin_window_attention_gb300 import capi
    case = st["case"]
    if case["op"] == "linear":
        y = capi.linear(st["x"], st["w"], st["b"], act=case["act"], residual=st["residual"], y=st["y"], pre=st["pre"])
        return [y] if st["pre"] is None else [y, st["pre"]]
    if case["op"] == "linear_bwd_data":
        return [capi.linear_bwd_data(st["dy"], st["w"], pre=st["pre"], act=case["act"], dx=st["dx"])]
    if case["op"] == "linear_bwd_weight":
        dw, db = capi.linear_bwd_weight(st["dy"], st["x"], dw=st["dw"], db=st["db"], workspace=st["workspace"])
        return [dw] if db is None else [dw, db]
    return [capi.orthogonalize(st["g"], steps=case["steps"], out=st["out"], workspace=st["workspace"])]


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * 0.7071067811865476))
                + z * torch.exp(-0.5 * z * z) * 0.3989422804014327)
    if act == "gelu_tanh":
        t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * 0.7978845608028654 * (1.0 + 0.134145 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _run_plain(st):
    case = st["case"]
    if case["op"] == "linear":
        z = st["x"].float() @ st["w"].float().t()
        if st["b"] is not None:
            z = z + st["b"]
        y = _act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        y = y.to(torch.bfloat16)
        return [y, z.to(torch.bfloat16)] if case["pre"] else [y]
    if case["op"] == "linear_bwd_data":
        d = st["dy"].float() @ st["w"].float()
        if case["act"] != "none":
            d = d * _act_grad(st["pre"].float(), case["act"])
        return [d.to(torch.bfloat16)]
    if case["op"] == "linear_bwd_weight":
        dy = st["dy"].float()
        dw = (dy.t() @ st["x"].float()).to(_DT[case["out"]])
        return [dw, dy.sum(0)] if case["bias"] else [dw]
    a, b, c = _NS
    x = st["g"].float()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
    tall = case["rows"] > case["cols"]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(case["steps"]):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if tall:
        x = x.transpose(1, 2)
    return [x.to(torch.bfloat16).contiguous()]


# ---- what a pass cannot do without -----------------------------------------------------

def work(case):
    if case["op"] == "orthogonalize":
        m, n = sorted((case["rows"], case["cols"]))
        elements = case["count"] * m * n
        # the Gram matrix and its square are symmetric: half of each product is enough
        flops = case["count"] * case["steps"] * (m * m * n + m ** 3 + 2 * m * m * n)
        return {"bytes": elements * ((2 if case["dtype"] == "bf16" else 4) + 2), "flops": flops}
    T, K, N = case["tokens"], case["K"], case["N"]
    flops = 2 * T * K * N
    if case["op"] == "linear":
        outs = T * N * (1 + int(case["residual"]) + int(case["pre"]))
        return {"bytes": 2 * (T * K + N * K + outs) + (4 * N if case["bias"] else 0), "flops": flops}
    if case["op"] == "linear_bwd_data":
        return {"bytes": 2 * (T * N + N * K + T * K * (1 if case["act"] == "none" else 2)), "flops": flops}
    return {"bytes": 2 * T * (N + K) + N * K * (4 if case["out"] == "fp32" else 2) + (4 * N if case["bias"] else 0),
            "flops": flops}


# ---- the definition in 64 bits -----------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "orthogonalize":
        a, b, c = _NS
        outs = []
        for g in st["g"]:
            x = g.to(d)
            x = x / (torch.linalg.vector_norm(x) + 1e-7)
            wide = x.shape[0] <= x.shape[1]
            for _ in range(case["steps"]):
                # the same odd polynomial of x, with the smaller Gram matrix on its own side
                if wide:
                    s = torch.mm(x, x.mT)
                    x = torch.mm(a * torch.eye(s.shape[0], dtype=d, device=s.device) + b * s + c * torch.mm(s, s), x)
                else:
                    s = torch.mm(x.mT, x)
                    x = torch.mm(x, a * torch.eye(s.shape[0], dtype=d, device=s.device) + b * s + c * torch.mm(s, s))
            outs.append(x)
        return [torch.stack(outs)]
    if case["op"] == "linear":
        z = torch.einsum("tk,nk->tn", st["x"].to(d), st["w"].to(d))
        if st["b"] is not None:
            z += st["b"].to(d)
        y = _exact_act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"].to(d)
        return [y, z] if case["pre"] else [y]
    if case["op"] == "linear_bwd_data":
        dx = torch.einsum("tn,nk->tk", st["dy"].to(d), st["w"].to(d))
        if case["act"] != "none":
            # the derivative by autograd of the fp64 activation
            z = st["pre"].to(d).requires_grad_(True)
            (slope,) = torch.autograd.grad(_exact_act(z, case["act"]).sum(), z)
            dx = dx * slope
        return [dx]
    dw = torch.einsum("tn,tk->nk", st["dy"].to(d), st["x"].to(d))
    return [dw, st["dy"].to(d).sum(0)] if case["bias"] else [dw]


def _exact_act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z
