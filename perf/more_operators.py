"""Operators around a block's products that are measured, with their plain forms.

What a Swin block needs beside its attention and its products, in training and in serving:

* ``block_norm``: the residual sum of a block with its gate, its stochastic depth and the norms
  before and after it; ``block_norm_bwd``: its gradients;
* ``GradClip``: the norm over all gradients of a model, and their clipping;
* ``quantize_fp4``, ``dequantize_fp4``: microscaled 4-bit operands (NVFP4: blocks of 16 with an
  E4M3 scale and a scale of the tensor, a power of two where it is not given; MXFP4: blocks of 32
  with a power of two), and back;
* ``linear_fp4``: a dense layer on such operands.

``run`` computes them in elementary torch operations in fp32, or, where ``own`` is set,
through the package's entry points; ``exact`` in fp64.
"""
import math

import torch

own = False

_DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---- cases -----------------------------------------------------------------------------

def _norm(op, T, C, kind="layer", block=True, pre=True, post=False, gate=False, samples=0, alpha=1.0, stream="bf16",
          dy=True):
    return {"op": op, "tokens": T, "C": C, "kind": kind, "block": block, "pre": pre, "post": post, "gate": gate,
            "samples": samples, "alpha": alpha, "stream": stream, "dy": dy}


def _clip(width, depths, window, classes, dtype, max_norm):
    return {"op": "clip", "width": width, "depths": depths, "window": window, "classes": classes, "dtype": dtype,
            "max_norm": max_norm}


def _round_trip(rows, K, fmt, dtype="bf16", std=1.0):
    return {"op": "round_trip", "rows": rows, "K": K, "format": fmt, "dtype": dtype, "std": std}


def _linear(T, K, N, fmt, act="none", bias=True, residual=False):
    return {"op": "linear_fp4", "tokens": T, "K": K, "N": N, "format": fmt, "act": act, "bias": bias,
            "residual": residual}


def listed():
    return [
        # the last norm of a served image's pooled token: latency counts
        dict(_norm("block_norm", 1, 1536, block=False), name="norm_one_token"),
        # between attention and MLP at the third stage: LayerScale, stochastic depth, the next norm;
        # a ragged number of tokens
        dict(_norm("block_norm", 12561, 768, gate=True, samples=3), name="norm_gate_ragged"),
        # a res-post-norm block at the first stage of 64 images, residual stream in fp32, and the
        # next block's norm
        dict(_norm("block_norm", 200704, 192, post=True, samples=64, stream="fp32"), name="norm_post_stage1"),
        # gradients of one window's tokens at the last stage, RMS norm
        dict(_norm("block_norm_bwd", 49, 1536, kind="rms", gate=True), name="norm_bwd_one_window"),
        # gradients at the first stage of 64 images, with norms on both sides, gate and depth
        dict(_norm("block_norm_bwd", 200704, 192, post=True, gate=True, samples=64), name="norm_bwd_stage1"),
        # the gradients of one small block: latency counts
        dict(_clip(96, "1", 7, 0, "fp32", 0.25), name="clip_one_block"),
        # the gradients of a large model, matrices in bf16 and vectors in fp32
        dict(_clip(192, "2-2-18-2", 7, 1000, "mixed", 5.0), name="clip_large_model"),
        # a wide weight to 4 bits and back, as for serving it
        dict(_round_trip(6144, 1536, "nvfp4", std=0.025), name="fp4_weight"),
        # activations of a ragged batch, fp32, odd width
        dict(_round_trip(12561, 1568, "mxfp4", dtype="fp32"), name="fp4_activations"),
        # the MLP's first product for one token
        dict(_linear(1, 1536, 6144, "nvfp4", act="gelu"), name="linear_fp4_one_token"),
        # the same for the tokens of one 224 image's last stage (one window)
        dict(_linear(49, 1536, 6144, "mxfp4", act="gelu"), name="linear_fp4_one_window"),
        # the MLP's second product with the shortcut, a ragged batch
        dict(_linear(12561, 6144, 1536, "nvfp4", residual=True), name="linear_fp4_fc2_ragged"),
    ]


_MAX_FLOPS = 2.3e11       # of a drawn product
_MAX_ELEMENTS = 3.8e7     # of a drawn operator's activations


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("block_norm", "block_norm_bwd", "clip", "round_trip", "linear_fp4", "linear_fp4"))
    if op in ("block_norm", "block_norm_bwd"):
        C = max(1, _log(rng, 8, 8192) // 8) * 8
        T = max(1, min(_log(rng, 1, 200704), int(_MAX_ELEMENTS / C)))
        block = rng.random() < 0.85
        pre = not block or rng.random() < 0.8
        samples = rng.choice((0, 1, 2, 3, 5, 16, 64)) if block else 0
        if samples:
            T = max(1, T // samples) * samples
        return _norm(op, T, C, rng.choice(("layer", "rms")), block, pre, block and rng.random() < 0.5,
                     block and rng.random() < 0.5, samples, rng.choice((1.0, 1.0, 2.5)) if block else 1.0,
                     rng.choice(("bf16", "fp32")), not pre or rng.random() < 0.8)
    if op == "clip":
        width = max(1, _log(rng, 32, 192) // 32) * 32
        depths = "-".join(str(rng.choice((1, 2, 6, 18) if i == 2 else (1, 2))) for i in range(rng.randint(1, 4)))
        return _clip(width, depths, rng.choice((4, 7, 12)), rng.choice((0, 10, 1000)),
                     rng.choice(("fp32", "bf16", "mixed")), rng.choice((0.5, 5.0, 1.0e4)))
    fmt = rng.choice(("nvfp4", "mxfp4"))
    if op == "round_trip":
        K = max(1, _log(rng, 32, 8192) // 32) * 32
        rows = max(1, min(_log(rng, 1, 50176), int(2.0e7 / K)))
        return _round_trip(rows, K, fmt, rng.choice(("bf16", "fp32")), rng.choice((1.0, 0.025, 40.0)))
    T, K, N = _log(rng, 1, 50176), max(1, _log(rng, 32, 8192) // 32) * 32, max(1, _log(rng, 8, 8192) // 8) * 8
    T = max(1, int(min(T, _MAX_FLOPS / (2.0 * K * N), 1.0e8 / (K + 2.0 * N))))
    return _linear(T, K, N, fmt, rng.choice(_ACTS), rng.random() < 0.8, rng.random() < 0.4)


# ---- inputs ----------------------------------------------------------------------------

def _grad_sizes(case):
    """Elements of every matrix and every vector gradient of a model: stages of doubling width, four
    norm vectors, a bias table, four matrices and their biases a block, a merging product between
    stages, a classifier."""
    mats, vecs = [], []
    depths = [int(d) for d in case["depths"].split("-")]
    for i, depth in enumerate(depths):
        c = case["width"] << i
        for _ in range(depth):
            mats += [3 * c * c, c * c, 4 * c * c, 4 * c * c]
            vecs += [c, c, 3 * c, (2 * case["window"] - 1) ** 2 * (c // 32), c, c, c, 4 * c, c]
        if i + 1 < len(depths):
            mats.append(8 * c * c)
            vecs += [4 * c, 4 * c]
    c = case["width"] << (len(depths) - 1)
    if case["classes"]:
        mats.append(case["classes"] * c)
        vecs += [case["classes"], c, c]
    return mats, vecs


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=_DEV, dtype=torch.float32) * std).to(dtype)

    def vector(n, mean=0.0, std=0.1):
        return normal(n, std=std, dtype=torch.float32) + mean

    st = {"case": case}
    if case["op"] in ("block_norm", "block_norm_bwd"):
        T, C, stream = case["tokens"], case["C"], _DT[case["stream"]]
        # the stream has a mean of its own in each channel, as after some blocks
        st["x"] = (normal(T, C, dtype=torch.float32) + vector(C, std=0.5)).to(stream)
        st["f"] = normal(T, C, std=0.7) if case["block"] else None
        st["pre"] = (vector(C, 1.0), vector(C) if case["kind"] == "layer" else None) if case["pre"] else None
        st["post"] = (vector(C, 1.0), vector(C) if case["kind"] == "layer" else None) if case["post"] else None
        st["gate"] = vector(C, 0.5, 0.2) if case["gate"] else None
        # stochastic depth: one sample in five is dropped, the others are scaled up
        n = case["samples"]
        st["keep"] = (torch.rand(n, generator=g, device=_DEV) < 0.8).float() / 0.8 if n else None
        if case["op"] == "block_norm_bwd":
            st["dh"] = normal(T, C, std=1e-3) if case["pre"] else None
            st["dy"] = normal(T, C, std=1e-3, dtype=stream) if case["dy"] else None
        if own and case["op"] == "block_norm_bwd":
            from swin_window_attention_gb300 import capi
            st["workspace"] = torch.empty(capi.swin_wattn_block_norm_bwd_workspace_bytes(T, C), dtype=torch.uint8,
                                          device=_DEV)
        return st
    if case["op"] == "clip":
        mats, vecs = _grad_sizes(case)
        dtypes = {"fp32": ("fp32", "fp32"), "bf16": ("bf16", "bf16"), "mixed": ("bf16", "fp32")}[case["dtype"]]
        # the gradients lie in one buffer a kind, one behind the other, whatever their sizes
        st["flat"] = [normal(sum(n), std=1e-3, dtype=_DT[d]) for n, d in zip((mats, vecs), dtypes)]
        st["out"] = [torch.empty_like(f) for f in st["flat"]]
        st["grads"] = [t for f, n in zip(st["flat"], (mats, vecs)) for t in torch.split(f, n)]
        st["clipped"] = [t for f, n in zip(st["out"], (mats, vecs)) for t in torch.split(f, n)]
        if own:
            from swin_window_attention_gb300 import capi
            st["clip"] = capi.GradClip(st["grads"], out=st["clipped"])
        return st
    if case["op"] == "round_trip":
        st["x"] = normal(case["rows"], case["K"], std=case["std"], dtype=_DT[case["dtype"]])
        return st
    T, K, N, fmt = case["tokens"], case["K"], case["N"], case["format"]
    st["x"] = normal(T, K)
    w = normal(N, K, std=K ** -0.5)
    st["b"] = vector(N) if case["bias"] else None
    st["residual"] = normal(T, N) if case["residual"] else None
    # of NVFP4 activations: a scale calibrated ahead of time, from the largest value of some batches
    st["x_scale"] = torch.full((1,), 4.8871 / 2688.0, device=_DEV) if fmt == "nvfp4" else None
    if own:
        from swin_window_attention_gb300 import capi
        st["w"] = capi.quantize_fp4(w, fmt)
    else:
        st["w"] = _round_trip_plain(w.float(), fmt, None)[0]
    return st


# ---- one pass --------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _given(*ts):
    return [t for t in ts if t is not None]


def _run_own(st):
    from swin_window_attention_gb300 import capi
    case = st["case"]
    if case["op"] == "block_norm":
        return _given(*capi.block_norm(st["x"], st["f"], pre=st["pre"], post=st["post"], gate=st["gate"],
                                       keep=st["keep"], alpha=case["alpha"], kind=case["kind"]))
    if case["op"] == "block_norm_bwd":
        dx, df, grads = capi.block_norm_bwd(st["x"], st["f"], dh=st["dh"], dy=st["dy"], pre=st["pre"], post=st["post"],
                                            gate=st["gate"], keep=st["keep"], alpha=case["alpha"], kind=case["kind"],
                                            workspace=st["workspace"])
        return _given(dx, df, *(grads.get(k) for k in ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate")))
    if case["op"] == "clip":
        norm = st["clip"](case["max_norm"])
        return [*st["out"], norm]
    if case["op"] == "round_trip":
        q = capi.quantize_fp4(st["x"], case["format"])
        return _given(capi.dequantize_fp4(q), q.tensor_scale)
    return [capi.linear_fp4(st["x"], st["w"], st["b"], act=case["act"], residual=st["residual"],
                            x_scale=st["x_scale"])]


def _normalised(v, kind):
    """v normalised over its last axis, and the factor."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = 1.0 / (v.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    return v * r, r


def _norm_slope(d, vhat, r, kind):
    """The gradient of a norm's input, for the gradient d of what it normalised to."""
    d = d - vhat * (d * vhat).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - d.mean(-1, keepdim=True)
    return d * r


def _affine(vhat, wb):
    v = vhat * wb[0]
    return v if wb[1] is None else v + wb[1]


def _of_tokens(keep, T):
    return keep.repeat_interleave(T // keep.numel()).unsqueeze(1)


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


def _tensor_scale(amax):
    """The smallest power of two of which amax is at most 6 * 448 = 2688 times."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), (e - torch.where(m > 0.65625, 11, 12)).clamp_min(-90))


def _round_trip_plain(x, fmt, scale):
    """x (fp32) to microscaled 4-bit values and back, and the scale of the tensor."""
    n = 16 if fmt == "nvfp4" else 32
    v = x.reshape(-1, n)
    amax = v.abs().amax(1, keepdim=True)
    if fmt == "nvfp4":
        ts = _tensor_scale(amax.amax().reshape(1)) if scale is None else scale
        s = (amax / 6.0 / ts).clamp_max(448.0).to(torch.float8_e4m3fn).float()
        step = s * ts
    else:
        ts, s = None, torch.ldexp(torch.ones_like(amax), (torch.frexp(amax)[1] - 3).clamp_min(-127))
        step = s
    q = (v / torch.where(step > 0, step, torch.ones_like(step))).abs().clamp_max(6.0)
    # the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; of two as near, the one whose last bit is 0
    gap = torch.where(q < 2.0, 0.5, torch.where(q < 4.0, 1.0, 2.0))
    q = torch.round(q / gap) * gap
    return (torch.copysign(q, v) * s * (1.0 if ts is None else ts)).reshape(x.shape), ts


def _run_plain(st):
    case = st["case"]
    if case["op"] == "block_norm":
        out, y = [], st["x"].float()
        if case["block"]:
            u = st["f"].float()
            if case["post"]:
                u = _affine(_normalised(u, case["kind"])[0], st["post"])
            if case["gate"]:
                u = u * st["gate"]
            if case["samples"]:
                u = u * _of_tokens(st["keep"], case["tokens"])
            y = case["alpha"] * y + u
            out.append(y.to(_DT[case["stream"]]))
        if case["pre"]:
            out.append(_affine(_normalised(y, case["kind"])[0], st["pre"]).to(torch.bfloat16))
        return out
    if case["op"] == "block_norm_bwd":
        grads = []
        d = st["dy"].float() if case["dy"] else 0.0
        if case["pre"]:
            dh = st["dh"].float()
            yhat, r = _normalised(st["x"].float(), case["kind"])
            grads.append((dh * yhat).sum(0))
            if case["kind"] == "layer":
                grads.append(dh.sum(0))
            d = d + _norm_slope(dh * st["pre"][0], yhat, r, case["kind"])
        out = [(case["alpha"] * d).to(_DT[case["stream"]])]
        if not case["block"]:
            return out + grads
        f = st["f"].float()
        if case["samples"]:
            d = d * _of_tokens(st["keep"], case["tokens"])
        u, dgate = f, None
        if case["post"]:
            fhat, r = _normalised(f, case["kind"])
            u = _affine(fhat, st["post"])
        if case["gate"]:
            dgate = (d * u).sum(0)
            d = d * st["gate"]
        if case["post"]:
            grads.append((d * fhat).sum(0))
            if case["kind"] == "layer":
                grads.append(d.sum(0))
            d = _norm_slope(d * st["post"][0], fhat, r, case["kind"])
        return out + [d.to(torch.bfloat16)] + grads + _given(dgate)
    if case["op"] == "clip":
        a, b = st["flat"]
        square = a.float().square().sum(dtype=torch.float64) + b.float().square().sum(dtype=torch.float64)
        norm = square.sqrt().float().reshape(1)
        factor = (case["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
        return [(a.float() * factor).to(a.dtype), (b.float() * factor).to(b.dtype), norm]
    if case["op"] == "round_trip":
        v, ts = _round_trip_plain(st["x"].float(), case["format"], None)
        return _given(v.to(torch.bfloat16), ts)
    z = _round_trip_plain(st["x"].float(), case["format"], st["x_scale"])[0] @ st["w"].t()
    if st["b"] is not None:
        z = z + st["b"]
    y = _act(z, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return [y.to(torch.bfloat16)]


# ---- what a pass cannot do without -----------------------------------------------------

def work(case):
    if case["op"] in ("block_norm", "block_norm_bwd"):
        n, stream, params = case["tokens"] * case["C"], 2 if case["stream"] == "bf16" else 4, case["C"] * 4
        vectors = (2 if case["kind"] == "layer" else 1) * (case["pre"] + case["post"]) + case["gate"]
        if case["op"] == "block_norm":
            per = stream + (2 + stream if case["block"] else 0) + (2 if case["pre"] else 0)
            return {"bytes": n * per + vectors * params, "flops": n * (6 * case["pre"] + 8 * case["post"] + 3)}
        # y, dh, dy, f in; dx, df out
        per = (stream + 2 if case["pre"] else 0) + (stream if case["dy"] else 0) + stream + (4 if case["block"] else 0)
        return {"bytes": n * per + 2 * vectors * params, "flops": n * (14 * case["pre"] + 18 * case["post"] + 4)}
    if case["op"] == "clip":
        mats, vecs = _grad_sizes(case)
        a, b = {"fp32": (4, 4), "bf16": (2, 2), "mixed": (2, 4)}[case["dtype"]]
        return {"bytes": 2 * (sum(mats) * a + sum(vecs) * b) + 4, "flops": 3 * (sum(mats) + sum(vecs))}
    nv = case["format"] == "nvfp4"
    packed = 0.5 + (1 / 16 if nv else 1 / 32)  # bytes of a 4-bit element with its share of a scale
    if case["op"] == "round_trip":
        n = case["rows"] * case["K"]
        return {"bytes": int(n * ((2 if case["dtype"] == "bf16" else 4) + 2 * packed + 2)), "flops": 4 * n}
    T, K, N = case["tokens"], case["K"], case["N"]
    return {"bytes": int(2 * T * K + packed * N * K + 2 * T * N * (1 + case["residual"]) + 4 * N * case["bias"]),
            "flops": 2 * T * K * N}


# ---- the definition in 64 bits -----------------------------------------------------------

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_scale(x):
    return torch.exp2(torch.ceil(torch.log2(x.abs().max() / 2688.0)))


def _exact_fp4(x, fmt, ts):
    """The values that x (fp64) stands for in 4 bits, by comparison with every one of them."""
    blocks = x.unflatten(-1, (-1, 16 if fmt == "nvfp4" else 32))
    top = blocks.abs().max(-1, keepdim=True).values
    if fmt == "nvfp4":
        ratio = (top / (6.0 * ts)).clamp(max=448.0)
        # E4M3: three bits behind the leading one, down to 2^-9
        ulp = torch.exp2(torch.floor(torch.log2(ratio.clamp(min=2.0 ** -6))) - 3)
        step = torch.round(ratio / ulp) * ulp * ts
    else:
        step = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2)
    v = blocks.abs() / torch.where(step > 0, step, 1.0)
    code = torch.zeros_like(v)
    for k in range(1, 8):
        middle = (_E2M1[k - 1] + _E2M1[k]) / 2
        # a middle goes to the neighbour of even number
        code = torch.where((v > middle) if k % 2 else (v >= middle), float(k), code)
    table = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    return (table[code.long()] * step * torch.sign(blocks)).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] in ("block_norm", "block_norm_bwd"):
        def norm(v, wb):
            if case["kind"] == "layer":
                v = v - v.mean(1, keepdim=True)
            v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-5) * wb[0]
            return v if wb[1] is None else v + wb[1]

        def pair(name):
            return None if st[name] is None else [None if p is None else p.to(d).requires_grad_(True) for p in st[name]]

        pre, post = pair("pre"), pair("post")
        gate = None if st["gate"] is None else st["gate"].to(d).requires_grad_(True)
        backward = case["op"] == "block_norm_bwd"
        x = st["x"].to(d)
        f = st["f"].to(d).requires_grad_(backward) if case["block"] else None
        branch = None
        if case["block"]:
            branch = f if post is None else norm(f, post)
            if gate is not None:
                branch = branch * gate
            if case["samples"]:
                branch = (branch.view(case["samples"], -1, case["C"]) * st["keep"].to(d).view(-1, 1, 1)).view_as(branch)
        if not backward:
            with torch.no_grad():
                y = x if branch is None else case["alpha"] * x + branch
                return ([] if branch is None else [y]) + ([] if pre is None else [norm(y, pre)])
        # the gradient of y by autograd through the pre-norm, then that of the block through it
        y = x.requires_grad_(True)
        total, pre_leaves = torch.zeros_like(x), [] if pre is None else _given(*pre)
        grads = []
        if pre is not None:
            got = torch.autograd.grad(norm(y, pre), [y, *pre_leaves], st["dh"].to(d))
            total, grads = total + got[0], list(got[1:])
        if st["dy"] is not None:
            total = total + st["dy"].to(d)
        out = [case["alpha"] * total]
        if branch is not None:
            leaves = [f] + ([] if post is None else _given(*post)) + _given(gate)
            got = torch.autograd.grad(branch, leaves, total)
            out, grads = out + [got[0]], grads + list(got[1:])
        return out + [t.detach() for t in grads]
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(torch.dot(c, c)) for f in st["flat"] for c in f.to(d).split(1 << 24)))
        factor = min(1.0, case["max_norm"] / (norm + 1e-6))
        return [*(f.to(d) * factor for f in st["flat"]), torch.tensor([norm], dtype=d)]
    if case["op"] == "round_trip":
        x = st["x"].to(d)
        if case["format"] == "mxfp4":
            return [_exact_fp4(x, "mxfp4", None)]
        ts = _exact_scale(x)
        return [_exact_fp4(x, "nvfp4", ts), ts.reshape(1)]
    z = torch.einsum("tk,nk->tn", _exact_fp4(st["x"].to(d), case["format"], st["x_scale"]), _exact_weight(case, seed))
    if st["b"] is not None:
        z += st["b"].to(d)
    y = _exact_act(z, case["act"])
    return [y if st["residual"] is None else y + st["residual"].to(d)]


def _exact_weight(case, seed):
    """The weight of the linear case, drawn as prepare does, as the 4-bit values it stands for."""
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    torch.randn(case["tokens"], case["K"], generator=g, device=_DEV, dtype=torch.float32)
    w = torch.randn(case["N"], case["K"], generator=g, device=_DEV, dtype=torch.float32) * case["K"] ** -0.5
    w = w.to(torch.bfloat16).to(torch.float64)
    return _exact_fp4(w, case["format"], _exact_scale(w))


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
