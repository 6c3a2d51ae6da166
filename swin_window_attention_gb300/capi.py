"""ctypes binding of libswin_wattn.so (declared in include/swin_wattn.h).

Argument marshalling only: every function forwards to the C entry point of the same
name and returns its status code; ``WindowAttention`` wraps a plan for torch CUDA
tensors. Every step of the computation runs in the library's CUDA kernels. If the
library has not been built (``python -m swin_window_attention_gb300.build``), ``load()``
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libswin_wattn.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_MISALIGNED = 3
ERR_BAD_PLAN = 4
ERR_CUDA = 5
ERR_TIMEOUT = 6
BF16 = 0
FP32 = 1
KERNEL_AUTO = 0
KERNEL_MMA_SYNC = 1
KERNEL_TCGEN05 = 2

ACT_NONE = 0
ACT_RELU = 1
ACT_GELU = 2
ACT_GELU_TANH = 3
ACT_SILU = 4
NORM_LAYER = 0
NORM_RMS = 1
NORMS = {"layer": NORM_LAYER, "rms": NORM_RMS}
NVFP4 = 0
MXFP4 = 1
FP4_FORMATS = {"nvfp4": NVFP4, "mxfp4": MXFP4}
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU}

# Every symbol include/swin_wattn.h declares, with (argtypes, restype).
_vp, _i, _cp = ctypes.c_void_p, ctypes.c_int, ctypes.c_char_p
SIGNATURES = {
    "swin_wattn_plan": ([ctypes.POINTER(_vp), _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp], _i),
    "swin_wattn_set_bias": ([_vp, _vp, _vp], _i),
    "swin_wattn_fwd": ([_vp, _vp, _vp, _vp], _i),
    "swin_wattn_fwd_host": ([_vp, _vp, _vp, _vp, _vp, _vp], _i),
    "swin_wattn_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp], _i),
    "swin_wattn_debug_maps": ([_vp, _vp, _vp, _vp, _vp, _vp], _i),
    "swin_wattn_bwd_noalloc": ([_vp, _vp, _vp, _vp, _vp] + [_i] * 8 + [_vp], _i),
    "swin_wattn_qkv_workspace_bytes": ([_i, _i], ctypes.c_size_t),
    "swin_wattn_qkv_proj": ([_vp] * 6 + [_i, _i, ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp], _i),
    "swin_wattn_qkv_prepared_bytes": ([_i], ctypes.c_size_t),
    "swin_wattn_qkv_stats_bytes": ([_i], ctypes.c_size_t),
    "swin_wattn_qkv_prepare": ([_vp] * 4 + [_i, _vp, ctypes.c_size_t, _vp], _i),
    "swin_wattn_qkv_proj_prepared": ([_vp] * 3 + [_i, _i, ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp], _i),
    "swin_wattn_qkv_proj_prepared_fp8": ([_vp] * 3 + [_i, _i] + [ctypes.c_float] * 4 +
                                         [_vp, _vp, ctypes.c_size_t, _vp, _vp], _i),
    "swin_wattn_proj_residual": ([_vp] * 5 + [_i, _i, _vp, _vp], _i),
    "swin_wattn_linear": ([_vp] * 6 + [_i] * 4 + [_vp, _vp], _i),
    "swin_wattn_linear_bwd_data": ([_vp] * 4 + [_i] * 4 + [_vp, _vp], _i),
    "swin_wattn_linear_bwd_weight_workspace_bytes": ([_i] * 3, ctypes.c_size_t),
    "swin_wattn_linear_bwd_weight": ([_vp] * 4 + [_i] * 5 + [_vp, ctypes.c_size_t, _vp, _vp], _i),
    "swin_wattn_orthogonalize_workspace_bytes": ([_i] * 3, ctypes.c_size_t),
    "swin_wattn_orthogonalize": ([_vp, _vp] + [_i] * 5 + [ctypes.c_float] * 2 + [_vp, ctypes.c_size_t, _vp, _vp], _i),
    "swin_wattn_block_norm": ([_vp] * 10 + [_i] * 5 + [ctypes.c_float] * 2 + [_vp], _i),
    "swin_wattn_block_norm_bwd_workspace_bytes": ([_i] * 2, ctypes.c_size_t),
    "swin_wattn_block_norm_bwd": ([_vp] * 16 + [_i] * 5 + [ctypes.c_float] * 2 + [_i, _vp, ctypes.c_size_t, _vp], _i),
    "swin_wattn_clip_list_bytes": ([_vp, _vp, _i], ctypes.c_size_t),
    "swin_wattn_clip_plan": ([ctypes.POINTER(_vp)] + [_vp] * 4 + [_i, _vp, ctypes.c_size_t, _vp], _i),
    "swin_wattn_clip_workspace_bytes": ([], ctypes.c_size_t),
    "swin_wattn_clip_grad_norm": ([_vp] + [ctypes.c_float] * 3 + [_vp, _vp, ctypes.c_size_t, _vp], _i),
    "swin_wattn_clip_destroy": ([_vp], _i),
    "swin_wattn_fp4_scale_bytes": ([_i] * 3, ctypes.c_size_t),
    "swin_wattn_fp4_workspace_bytes": ([], ctypes.c_size_t),
    "swin_wattn_fp4_quantize": ([_vp] * 4 + [_i] * 5 + [_vp, ctypes.c_size_t, _vp], _i),
    "swin_wattn_fp4_dequantize": ([_vp] * 4 + [_i] * 4 + [_vp], _i),
    "swin_wattn_linear_fp4": ([_vp] * 9 + [_i] * 5 + [_vp, _vp], _i),
    "swin_wattn_linear_fp4_workspace_bytes": ([_i] * 5, ctypes.c_size_t),
    "swin_wattn_linear_fp4_of": ([_vp] * 8 + [_i] * 6 + [_vp, ctypes.c_size_t, _vp, _vp], _i),
    "swin_wattn_fwd_fp8": ([_vp, _vp, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp], _i),
    "swin_wattn_set_fwd_kernel": ([_vp, _i], _i),
    "swin_wattn_fwd_kernel": ([_vp], _i),
    "swin_wattn_set_bwd_kernel": ([_vp, _i], _i),
    "swin_wattn_bwd_kernel": ([_vp], _i),
    "swin_wattn_device_status": ([_vp, _vp], _i),
    "swin_wattn_destroy": ([_vp], _i),
    "swin_wattn_status_string": ([_i], _cp),
    "swin_wattn_last_error": ([], _cp),
    "swin_wattn_launch_count": ([_i], ctypes.c_uint64),
}

# The fault-injection library (include/swin_wattn_debug.h) adds one entry point.
DEBUG_LIB_PATH = os.path.join(_HERE, "libswin_wattn_debug.so")
DEBUG_SIGNATURES = {"swin_wattn_debug_set_fault": ([_i, ctypes.c_int64], _i)}
FAULT_NONE = 0
FAULT_FWD_MMA_SYNC = 1
FAULT_FWD_TCGEN05 = 2
FAULT_GEMM = 3

_lib = None
_debug_lib = None


class SwinWAttnError(RuntimeError):
    def __init__(self, where: str, status: int):
        lib = load()
        msg = lib.swin_wattn_status_string(status).decode()
        if status == ERR_CUDA:
            msg += ": " + lib.swin_wattn_last_error().decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m swin_window_attention_gb300.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def load_debug() -> ctypes.CDLL:
    """Load the fault-injection build (once), a separate library with the same entry
    points plus swin_wattn_debug_set_fault. Raises if it has not been built
    (``python -m swin_window_attention_gb300.build --debug``)."""
    global _debug_lib
    if _debug_lib is None:
        if not os.path.exists(DEBUG_LIB_PATH):
            raise RuntimeError(f"{DEBUG_LIB_PATH} is missing: build it with "
                               "`python -m swin_window_attention_gb300.build --debug`")
        lib = ctypes.CDLL(DEBUG_LIB_PATH)
        for name, (args, res) in list(SIGNATURES.items()) + list(DEBUG_SIGNATURES.items()):
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _debug_lib = lib
    return _debug_lib


# ---- same names as the C entry points --------------------------------------------------

def swin_wattn_plan(B, H, W, C, num_heads, window, shift, dtype, bias_table_ptr, stream):
    """Returns (status, plan handle or None)."""
    h = _vp()
    rc = load().swin_wattn_plan(ctypes.byref(h), B, H, W, C, num_heads, window, shift, dtype,
                                bias_table_ptr, stream)
    return rc, (h.value if rc == OK else None)


def swin_wattn_set_bias(plan, bias_table_ptr, stream):
    return load().swin_wattn_set_bias(plan, bias_table_ptr, stream)


def swin_wattn_fwd(plan, qkv_ptr, out_ptr, stream):
    return load().swin_wattn_fwd(plan, qkv_ptr, out_ptr, stream)


def swin_wattn_fwd_host(plan, qkv_host_ptr, out_host_ptr, dev_qkv_ptr, dev_out_ptr, stream):
    return load().swin_wattn_fwd_host(plan, qkv_host_ptr, out_host_ptr, dev_qkv_ptr,
                                      dev_out_ptr, stream)


def swin_wattn_bwd(plan, qkv_ptr, dout_ptr, dqkv_ptr, dtable_ptr, stream):
    return load().swin_wattn_bwd(plan, qkv_ptr, dout_ptr, dqkv_ptr, dtable_ptr, stream)


def swin_wattn_debug_maps(plan, gather_ptr, relidx_ptr, mask_ptr, dense_bias_ptr, stream):
    return load().swin_wattn_debug_maps(plan, gather_ptr, relidx_ptr, mask_ptr, dense_bias_ptr,
                                        stream)


def swin_wattn_bwd_noalloc(qkv_ptr, dout_ptr, dqkv_ptr, dtable_ptr, table_ptr, B, H, W, C,
                           num_heads, window, shift, dtype, stream):
    """Backward with no plan and no device allocation (fixed working memory in the
    library); see include/swin_wattn.h."""
    return load().swin_wattn_bwd_noalloc(qkv_ptr, dout_ptr, dqkv_ptr, dtable_ptr, table_ptr, B, H,
                                         W, C, num_heads, window, shift, dtype, stream)


def swin_wattn_qkv_workspace_bytes(C, tokens):
    return int(load().swin_wattn_qkv_workspace_bytes(C, tokens))


def swin_wattn_qkv_proj(x_ptr, gamma_ptr, beta_ptr, w_ptr, b_ptr, qkv_ptr, tokens, C, eps, workspace_ptr,
                        workspace_bytes, status_ptr, stream):
    return load().swin_wattn_qkv_proj(x_ptr, gamma_ptr, beta_ptr, w_ptr, b_ptr, qkv_ptr, tokens, C, eps,
                                      workspace_ptr, workspace_bytes, status_ptr, stream)


def qkv_proj(x, gamma, beta, w, b, qkv=None, eps=1e-5, status=None, workspace=None, stream=None):
    """LayerNorm over the last axis of the bf16 CUDA tensor x [..., C], then x W^T + b into
    a bf16 [..., 3C] tensor (allocated here when not given; so is the workspace)."""
    import torch
    C = x.shape[-1]
    if qkv is None:
        qkv = torch.empty(x.shape[:-1] + (3 * C,), dtype=torch.bfloat16, device=x.device)
    tokens = x.numel() // C
    if workspace is None:
        workspace = torch.empty(max(swin_wattn_qkv_workspace_bytes(C, tokens), 1), dtype=torch.uint8,
                                device=x.device)
    rc = swin_wattn_qkv_proj(x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), w.data_ptr(), b.data_ptr(),
                             qkv.data_ptr(), tokens, C, eps, workspace.data_ptr(), workspace.numel(),
                             None if status is None else status.data_ptr(), _stream_handle(stream))
    if rc != OK:
        raise SwinWAttnError("swin_wattn_qkv_proj", rc)
    return qkv


def swin_wattn_qkv_prepared_bytes(C):
    return int(load().swin_wattn_qkv_prepared_bytes(C))


def swin_wattn_qkv_stats_bytes(tokens):
    return int(load().swin_wattn_qkv_stats_bytes(tokens))


def swin_wattn_qkv_prepare(gamma_ptr, beta_ptr, w_ptr, b_ptr, C, prepared_ptr, prepared_bytes, stream):
    return load().swin_wattn_qkv_prepare(gamma_ptr, beta_ptr, w_ptr, b_ptr, C, prepared_ptr, prepared_bytes, stream)


def swin_wattn_qkv_proj_prepared(x_ptr, prepared_ptr, qkv_ptr, tokens, C, eps, stats_ptr, stats_bytes, status_ptr,
                                 stream):
    return load().swin_wattn_qkv_proj_prepared(x_ptr, prepared_ptr, qkv_ptr, tokens, C, eps, stats_ptr,
                                               stats_bytes, status_ptr, stream)


class QkvProjection:
    """The producer step with its weights prepared once: LayerNorm over the last axis of a
    bf16 CUDA tensor x [..., C], then x W^T + b, for fixed gamma, beta, W [3C, C], b [3C]."""

    def __init__(self, gamma, beta, w, b, stream=None):
        import torch
        self.C = int(w.shape[1])
        self.prepared = torch.empty(max(swin_wattn_qkv_prepared_bytes(self.C), 1), dtype=torch.uint8,
                                    device=w.device)
        rc = swin_wattn_qkv_prepare(gamma.data_ptr(), beta.data_ptr(), w.data_ptr(), b.data_ptr(), self.C,
                                    self.prepared.data_ptr(), self.prepared.numel(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_qkv_prepare", rc)
        self.stats = None

    def __call__(self, x, qkv=None, eps=1e-5, status=None, stream=None):
        import torch
        C = self.C
        tokens = x.numel() // C
        if qkv is None:
            qkv = torch.empty(x.shape[:-1] + (3 * C,), dtype=torch.bfloat16, device=x.device)
        need = max(swin_wattn_qkv_stats_bytes(tokens), 16)
        if self.stats is None or self.stats.numel() < need:
            self.stats = torch.empty(need, dtype=torch.uint8, device=x.device)
        rc = swin_wattn_qkv_proj_prepared(x.data_ptr(), self.prepared.data_ptr(), qkv.data_ptr(), tokens, C, eps,
                                          self.stats.data_ptr(), self.stats.numel(),
                                          None if status is None else status.data_ptr(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_qkv_proj_prepared", rc)
        return qkv

    def fp8(self, x, scales, qkv8=None, amax=None, eps=1e-5, status=None, stream=None):
        """The same projection with OCP FP8 E4M3 output, qkv8 = E4M3(qkv / scale_t) for the
        tensor t (q, k, v) of each channel, as a uint8 [..., 3C] tensor (allocated here when
        not given); amax, an optional CUDA float tensor [3], receives max |qkv_t| (max-ed)."""
        import torch
        C = self.C
        tokens = x.numel() // C
        if qkv8 is None:
            qkv8 = torch.empty(x.shape[:-1] + (3 * C,), dtype=torch.uint8, device=x.device)
        need = max(swin_wattn_qkv_stats_bytes(tokens), 16)
        if self.stats is None or self.stats.numel() < need:
            self.stats = torch.empty(need, dtype=torch.uint8, device=x.device)
        sq, sk, sv = (float(v) for v in scales)
        rc = swin_wattn_qkv_proj_prepared_fp8(x.data_ptr(), self.prepared.data_ptr(), qkv8.data_ptr(), tokens, C,
                                              eps, sq, sk, sv, None if amax is None else amax.data_ptr(),
                                              self.stats.data_ptr(), self.stats.numel(),
                                              None if status is None else status.data_ptr(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_qkv_proj_prepared_fp8", rc)
        return qkv8


def swin_wattn_qkv_proj_prepared_fp8(x_ptr, prepared_ptr, qkv8_ptr, tokens, C, eps, scale_q, scale_k, scale_v,
                                     amax_ptr, stats_ptr, stats_bytes, status_ptr, stream):
    return load().swin_wattn_qkv_proj_prepared_fp8(x_ptr, prepared_ptr, qkv8_ptr, tokens, C, eps, scale_q, scale_k,
                                                   scale_v, amax_ptr, stats_ptr, stats_bytes, status_ptr, stream)


def swin_wattn_proj_residual(o_ptr, wp_ptr, bp_ptr, residual_ptr, y_ptr, tokens, C, status_ptr, stream):
    return load().swin_wattn_proj_residual(o_ptr, wp_ptr, bp_ptr, residual_ptr, y_ptr, tokens, C, status_ptr,
                                           stream)


def proj_residual(o, wp, bp, residual, y=None, status=None, stream=None):
    """residual + o Wp^T + bp over the last axis of the bf16 CUDA tensors o and residual
    [..., C] into a bf16 [..., C] tensor (allocated here when not given; it may be the
    residual itself)."""
    import torch
    C = o.shape[-1]
    if y is None:
        y = torch.empty(o.shape, dtype=torch.bfloat16, device=o.device)
    rc = swin_wattn_proj_residual(o.data_ptr(), wp.data_ptr(), bp.data_ptr(), residual.data_ptr(), y.data_ptr(),
                                  o.numel() // C, C, None if status is None else status.data_ptr(),
                                  _stream_handle(stream))
    if rc != OK:
        raise SwinWAttnError("swin_wattn_proj_residual", rc)
    return y


def swin_wattn_linear(x_ptr, w_ptr, b_ptr, residual_ptr, y_ptr, pre_ptr, tokens, K, N, act, status_ptr, stream):
    return load().swin_wattn_linear(x_ptr, w_ptr, b_ptr, residual_ptr, y_ptr, pre_ptr, tokens, K, N, act, status_ptr,
                                    stream)


def swin_wattn_linear_bwd_data(dy_ptr, w_ptr, pre_ptr, dx_ptr, tokens, K, N, act, status_ptr, stream):
    return load().swin_wattn_linear_bwd_data(dy_ptr, w_ptr, pre_ptr, dx_ptr, tokens, K, N, act, status_ptr, stream)


def swin_wattn_linear_bwd_weight_workspace_bytes(tokens, K, N):
    return int(load().swin_wattn_linear_bwd_weight_workspace_bytes(tokens, K, N))


def swin_wattn_linear_bwd_weight(dy_ptr, x_ptr, dw_ptr, db_ptr, tokens, K, N, dtype, accumulate, workspace_ptr,
                                 workspace_bytes, status_ptr, stream):
    return load().swin_wattn_linear_bwd_weight(dy_ptr, x_ptr, dw_ptr, db_ptr, tokens, K, N, dtype, accumulate,
                                               workspace_ptr, workspace_bytes, status_ptr, stream)


def swin_wattn_orthogonalize_workspace_bytes(count, rows, cols):
    return int(load().swin_wattn_orthogonalize_workspace_bytes(count, rows, cols))


def swin_wattn_orthogonalize(g_ptr, out_ptr, count, rows, cols, dtype, steps, eps, scale, workspace_ptr,
                             workspace_bytes, status_ptr, stream):
    return load().swin_wattn_orthogonalize(g_ptr, out_ptr, count, rows, cols, dtype, steps, eps, scale, workspace_ptr,
                                           workspace_bytes, status_ptr, stream)


def swin_wattn_block_norm(x_ptr, f_ptr, pre_w_ptr, pre_b_ptr, post_w_ptr, post_b_ptr, gate_ptr, keep_ptr, y_ptr, h_ptr,
                          tokens, C, samples, dtype, kind, alpha, eps, stream):
    return load().swin_wattn_block_norm(x_ptr, f_ptr, pre_w_ptr, pre_b_ptr, post_w_ptr, post_b_ptr, gate_ptr, keep_ptr,
                                        y_ptr, h_ptr, tokens, C, samples, dtype, kind, alpha, eps, stream)


def swin_wattn_block_norm_bwd_workspace_bytes(tokens, C):
    return int(load().swin_wattn_block_norm_bwd_workspace_bytes(tokens, C))


def swin_wattn_block_norm_bwd(y_ptr, f_ptr, dh_ptr, dy_ptr, pre_w_ptr, post_w_ptr, post_b_ptr, gate_ptr, keep_ptr, dx_ptr,
                              df_ptr, dpre_w_ptr, dpre_b_ptr, dpost_w_ptr, dpost_b_ptr, dgate_ptr, tokens, C, samples,
                              dtype, kind, alpha, eps, accumulate, workspace_ptr, workspace_bytes, stream):
    return load().swin_wattn_block_norm_bwd(y_ptr, f_ptr, dh_ptr, dy_ptr, pre_w_ptr, post_w_ptr, post_b_ptr, gate_ptr,
                                            keep_ptr, dx_ptr, df_ptr, dpre_w_ptr, dpre_b_ptr, dpost_w_ptr, dpost_b_ptr,
                                            dgate_ptr, tokens, C, samples, dtype, kind, alpha, eps, accumulate,
                                            workspace_ptr, workspace_bytes, stream)


def swin_wattn_clip_list_bytes(sizes, dtypes):
    n = len(sizes)
    return int(load().swin_wattn_clip_list_bytes((ctypes.c_int64 * n)(*sizes), (_i * n)(*dtypes), n))


def swin_wattn_clip_plan(grad_ptrs, out_ptrs, sizes, dtypes, list_ptr, list_bytes, stream):
    """Returns (status, plan handle or None) for lists of device pointers, sizes and dtype codes."""
    n, h = len(grad_ptrs), _vp()
    rc = load().swin_wattn_clip_plan(ctypes.byref(h), (_vp * n)(*grad_ptrs), (_vp * n)(*out_ptrs),
                                     (ctypes.c_int64 * n)(*sizes), (_i * n)(*dtypes), n, list_ptr, list_bytes, stream)
    return rc, (h.value if rc == OK else None)


def swin_wattn_clip_workspace_bytes():
    return int(load().swin_wattn_clip_workspace_bytes())


def swin_wattn_clip_grad_norm(plan, max_norm, scale, eps, norm_ptr, workspace_ptr, workspace_bytes, stream):
    return load().swin_wattn_clip_grad_norm(plan, max_norm, scale, eps, norm_ptr, workspace_ptr, workspace_bytes, stream)


def swin_wattn_clip_destroy(plan):
    return load().swin_wattn_clip_destroy(plan)


def swin_wattn_fp4_scale_bytes(rows, K, format):
    return int(load().swin_wattn_fp4_scale_bytes(rows, K, format))


def swin_wattn_fp4_workspace_bytes():
    return int(load().swin_wattn_fp4_workspace_bytes())


def swin_wattn_fp4_quantize(x_ptr, codes_ptr, scales_ptr, tensor_scale_ptr, rows, K, format, dtype, scale_given,
                            workspace_ptr, workspace_bytes, stream):
    return load().swin_wattn_fp4_quantize(x_ptr, codes_ptr, scales_ptr, tensor_scale_ptr, rows, K, format, dtype,
                                          scale_given, workspace_ptr, workspace_bytes, stream)


def swin_wattn_fp4_dequantize(codes_ptr, scales_ptr, tensor_scale_ptr, out_ptr, rows, K, format, dtype, stream):
    return load().swin_wattn_fp4_dequantize(codes_ptr, scales_ptr, tensor_scale_ptr, out_ptr, rows, K, format, dtype, stream)


def swin_wattn_linear_fp4(x_codes_ptr, x_scales_ptr, x_tensor_scale_ptr, w_codes_ptr, w_scales_ptr, w_tensor_scale_ptr,
                          b_ptr, residual_ptr, y_ptr, tokens, K, N, format, act, status_ptr, stream):
    return load().swin_wattn_linear_fp4(x_codes_ptr, x_scales_ptr, x_tensor_scale_ptr, w_codes_ptr, w_scales_ptr,
                                        w_tensor_scale_ptr, b_ptr, residual_ptr, y_ptr, tokens, K, N, format, act,
                                        status_ptr, stream)


def swin_wattn_linear_fp4_workspace_bytes(tokens, K, N, format, scale_given):
    return int(load().swin_wattn_linear_fp4_workspace_bytes(tokens, K, N, format, scale_given))


def swin_wattn_linear_fp4_of(x_ptr, x_tensor_scale_ptr, w_codes_ptr, w_scales_ptr, w_tensor_scale_ptr, b_ptr, residual_ptr,
                             y_ptr, tokens, K, N, format, dtype, act, workspace_ptr, workspace_bytes, status_ptr, stream):
    return load().swin_wattn_linear_fp4_of(x_ptr, x_tensor_scale_ptr, w_codes_ptr, w_scales_ptr, w_tensor_scale_ptr, b_ptr,
                                           residual_ptr, y_ptr, tokens, K, N, format, dtype, act, workspace_ptr,
                                           workspace_bytes, status_ptr, stream)


# The wrappers of the MLP's products and the weight update check their tensors: a small product
# is over in a few microseconds, so the checks compare attributes first and look for the
# reason only when one differs.

_BF16 = torch.bfloat16
_F32 = torch.float32
_U8 = torch.uint8


def _address(name, t, shape, dtype, dev):
    """The address of one operand, checked: a contiguous CUDA tensor of the given shape and
    dtype on CUDA device number `dev`."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name} is not contiguous")


def _plain(name, t, dtype, dev):
    """The same of an operand whose shape its caller has looked at."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _address(name, t, t.shape, dtype, dev)


def _leading(shape, width):
    """The axes before the last of an operand, as sizes of a result that ends in `width`, and how
    many rows they make."""
    if len(shape) == 2:
        return shape[0], (shape[0], width)
    return shape[:-1].numel(), (*shape[:-1], width)


def _device_of(name, t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} is not a CUDA tensor")
    return dev


def _float_code(name, t):
    """FP32 or BF16 for a tensor that may be either."""
    if t.dtype is _F32:
        return FP32
    if t.dtype is _BF16:
        return BF16
    raise ValueError(f"{name} has dtype {t.dtype}, not {_F32} or {_BF16}")


_INT_MAX = 0x7fffffff  # the C functions take sizes as ints: a larger one would arrive cut


def _too_large(*sizes):
    return ValueError(f"sizes {sizes}: none may be above 2^31 - 1")


_one_device = None  # whether the process sees a single device, which then is the current one


def _is_current(dev):
    global _one_device
    if _one_device is None:
        _one_device = torch.cuda.device_count() == 1
    return _one_device or dev == torch._C._cuda_getDevice()


def _call(fn, dev, stream, status, *args):
    """The C function fn(*args, status, stream) with device number `dev` current, on `stream`
    or that device's current stream; raises on an error status."""
    st = None if status is None else _address("status", status, (1,), torch.int32, dev)
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if _one_device or _is_current(dev):
        rc = fn(*args, st, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st, handle)
    if rc != OK:
        raise SwinWAttnError(fn.__name__, rc)


def _empty(shape, dtype, dev, stream):
    """A tensor of `stream`'s own memory pool (of the device's current stream without one),
    so that it may be used and freed in that stream's order."""
    device = _devices.get(dev) or _new_device(dev)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _vectors(n, size, dev, stream):
    """n fp32 vectors, each as _empty makes it. (Views of one allocation take half as long again.)"""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _vectors(n, size, dev, None)
    device = _devices.get(dev) or _new_device(dev)
    return [torch.empty(size, dtype=_F32, device=device) for _ in range(n)]


def _new_device(dev):
    return _devices.setdefault(dev, torch.device("cuda", dev))


_devices = {}  # by number: torch takes two microseconds longer for a number


def _act_code(act):
    code = ACTIVATIONS.get(act) if type(act) is str else act
    if code is None or not ACT_NONE <= code <= ACT_SILU:
        raise ValueError(f"unknown activation {act!r}: one of {sorted(ACTIVATIONS)} or an ACT_ code")
    return code


def _widths(name, shape, w, axis):
    """N and K of the weight [N, K], `axis` of which is the last of the operand `name`."""
    ws = w.shape
    if len(ws) != 2:
        raise ValueError(f"w has {len(ws)} dimensions, not 2")
    if not shape or shape[-1] != ws[axis]:
        raise ValueError(f"{name} has shape {tuple(shape)}, whose last axis does not fit w's {tuple(ws)}")
    return ws


def linear(x, w, b=None, act=ACT_NONE, residual=None, y=None, pre=None, status=None, stream=None):
    """residual + act(x W^T + b) over the last axis of the bf16 CUDA tensor x [..., K] with
    W [N, K] bf16 and b [N] fp32 (or None), into a bf16 [..., N] tensor (allocated here when
    not given; it may be the residual itself). act: "none", "relu", "gelu", "gelu_tanh",
    "silu" or an ACT_ code. pre, a bf16 [..., N] tensor, receives x W^T + b for the backward."""
    dev, xs = _device_of("x", x), x.shape
    N, K = _widths("x", xs, w, 1)
    tokens, shape = _leading(xs, N)
    if tokens > _INT_MAX or K > _INT_MAX or N > _INT_MAX:
        raise _too_large(tokens, K, N)
    if y is None:
        y = _empty(shape, _BF16, dev, stream)
    _call((_lib or load()).swin_wattn_linear, dev, stream, status, _plain("x", x, _BF16, dev), _plain("w", w, _BF16, dev),
          None if b is None else _address("b", b, (N,), _F32, dev),
          None if residual is None else _address("residual", residual, shape, _BF16, dev),
          _address("y", y, shape, _BF16, dev), None if pre is None else _address("pre", pre, shape, _BF16, dev),
          tokens, K, N, _act_code(act))
    return y


def linear_bwd_data(dy, w, pre=None, act=ACT_NONE, dx=None, status=None, stream=None):
    """(dy W) * act'(pre) for dy [..., N] and W [N, K], into a bf16 [..., K] tensor (allocated
    here when not given; it may be pre itself): with act "none" the gradient of the product's
    input, else of the pre-activation [..., K] whose activation that input was."""
    dev, ds = _device_of("dy", dy), dy.shape
    code = _act_code(act)
    N, K = _widths("dy", ds, w, 0)
    tokens, shape = _leading(ds, K)
    if tokens > _INT_MAX or K > _INT_MAX or N > _INT_MAX:
        raise _too_large(tokens, K, N)
    if code != ACT_NONE and pre is None:
        raise ValueError("an activation needs its pre-activation: pre is None")
    if dx is None:
        dx = _empty(shape, _BF16, dev, stream)
    _call((_lib or load()).swin_wattn_linear_bwd_data, dev, stream, status, _plain("dy", dy, _BF16, dev),
          _plain("w", w, _BF16, dev), None if pre is None else _address("pre", pre, shape, _BF16, dev),
          _address("dx", dx, shape, _BF16, dev), tokens, K, N, code)
    return dx


def linear_bwd_weight(dy, x, dw=None, db=None, accumulate=False, workspace=None, status=None, stream=None):
    """dW = dy^T x [N, K] and db = the sum of dy over the tokens, for dy [..., N] and
    x [..., K]. dw (fp32 or bf16) and db (fp32) are the tensors to write, or with accumulate
    to add to; without dw both are allocated here, in fp32; with dw alone there is no db.
    workspace: a uint8 tensor of swin_wattn_linear_bwd_weight_workspace_bytes (allocated here
    when not given). Returns (dw, db)."""
    dev, ds, xs = _device_of("dy", dy), dy.shape, x.shape
    if not ds or not xs or ds[:-1] != xs[:-1]:
        raise ValueError(f"dy and x have shapes {tuple(ds)} and {tuple(xs)}: they differ before the last axis")
    N, K = ds[-1], xs[-1]
    tokens = ds[0] if len(ds) == 2 else ds[:-1].numel()
    if tokens > _INT_MAX or K > _INT_MAX or N > _INT_MAX:
        raise _too_large(tokens, K, N)
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs the dw to add to")
        dw = _empty((N, K), _F32, dev, stream)
        db = _empty((N,), _F32, dev, stream) if db is None else db
    code = _float_code("dw", dw)
    if workspace is None:
        workspace = _empty((max(swin_wattn_linear_bwd_weight_workspace_bytes(tokens, K, N), 1),), _U8, dev, stream)
    _call((_lib or load()).swin_wattn_linear_bwd_weight, dev, stream, status, _plain("dy", dy, _BF16, dev),
          _plain("x", x, _BF16, dev), _address("dw", dw, (N, K), dw.dtype, dev),
          None if db is None else _address("db", db, (N,), _F32, dev), tokens, K, N, code, 1 if accumulate else 0,
          _plain("workspace", workspace, _U8, dev), workspace.numel())
    return dw, db


def orthogonalize(g, steps=5, eps=1e-7, scale=1.0, out=None, workspace=None, status=None, stream=None):
    """scale * X after `steps` Newton-Schulz steps from X = G / (|G| + eps) for each matrix of
    the fp32 or bf16 CUDA tensor g [rows, cols] or [count, rows, cols], into a bf16 tensor of
    its shape (allocated here when not given). workspace: a uint8 tensor of
    swin_wattn_orthogonalize_workspace_bytes (allocated here when not given)."""
    dev = _device_of("g", g)
    shape, code = g.shape, _float_code("g", g)
    if len(shape) not in (2, 3):
        raise ValueError(f"g has {len(shape)} dimensions, not 2 or 3")
    count, rows, cols = (1, *shape) if len(shape) == 2 else shape
    steps = int(steps)
    if count > _INT_MAX or rows > _INT_MAX or cols > _INT_MAX or abs(steps) > _INT_MAX:
        raise _too_large(count, rows, cols, steps)
    if out is None:
        out = _empty(shape, _BF16, dev, stream)
    if workspace is None:
        workspace = _empty((max(swin_wattn_orthogonalize_workspace_bytes(count, rows, cols), 1),), _U8, dev, stream)
    _call((_lib or load()).swin_wattn_orthogonalize, dev, stream, status, _plain("g", g, g.dtype, dev),
          _address("out", out, shape, _BF16, dev), count, rows, cols, code, steps, float(eps), float(scale),
          _plain("workspace", workspace, _U8, dev), workspace.numel())
    return out


def _launch(fn, dev, stream, *args):
    """The C function fn(*args, stream) as _call runs it, for those that take no status word."""
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if _one_device or _is_current(dev):
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != OK:
        raise SwinWAttnError(fn.__name__, rc)


def _kind_code(kind):
    code = NORMS.get(kind) if type(kind) is str else kind
    if code is None or not NORM_LAYER <= code <= NORM_RMS:
        raise ValueError(f"unknown norm {kind!r}: one of {sorted(NORMS)} or a NORM_ code")
    return code


def _vector(name, t, n, dev):
    """The address of an fp32 vector of n values."""
    return _address(name, t, (n,), _F32, dev)


def _block_shape(shape, f, post, gate, keep, alpha):
    """Sizes of a block_norm call, checked: tokens, C, samples."""
    if not shape:
        raise ValueError("x has no dimensions")
    C = shape[-1]
    tokens = shape[0] if len(shape) == 2 else shape[:-1].numel()
    if tokens > _INT_MAX or C > _INT_MAX:
        raise _too_large(tokens, C)
    if f is None and not (post is None and gate is None and keep is None and alpha == 1.0):
        raise ValueError("post, gate, keep and alpha belong to a block: f is None")
    if keep is None:
        return tokens, C, 0
    samples = keep.numel()
    if samples < 1 or tokens % samples:
        raise ValueError(f"keep has {samples} samples, which do not divide {tokens} tokens")
    return tokens, C, samples


def block_norm(x, f=None, pre=None, post=None, gate=None, keep=None, alpha=1.0, kind="layer", eps=1e-5, y=None, h=None,
               stream=None):
    """The residual sum around a block and the norms on both sides: with u = post(f) (f without
    post), y = alpha x + keep[sample] gate[channel] u and h = pre(y). x [..., C] is the residual
    stream, a bf16 or fp32 CUDA tensor, f the block's output in bf16. pre and post: (weight, bias)
    of the norm before the next block and after this one, fp32 [C], the bias may be None; gate fp32
    [C]; keep fp32 [samples], for equal runs of tokens (stochastic depth). kind: "layer" or "rms".
    Returns (y, h), y of x's dtype (into y, which may be x itself) or None without f, h in bf16 or
    None without pre."""
    dev, shape, dtype = _device_of("x", x), x.shape, x.dtype
    tokens, C, samples = _block_shape(shape, f, post, gate, keep, alpha)
    code = _float_code("x", x)
    pf = py = ph = pre_w = pre_b = post_w = post_b = None
    if f is not None:
        pf = _address("f", f, shape, _BF16, dev)
        if y is None:
            y = _empty(shape, dtype, dev, stream)
            py = y.data_ptr()
        else:
            py = _address("y", y, shape, dtype, dev)
    elif pre is None:
        raise ValueError("neither f nor pre is given: there is nothing to do")
    elif y is not None:
        raise ValueError("y needs f")
    if pre is not None:
        w, b = pre
        pre_w = _vector("pre weight", w, C, dev)
        if b is not None:
            pre_b = _vector("pre bias", b, C, dev)
        if h is None:
            h = _empty(shape, _BF16, dev, stream)
            ph = h.data_ptr()
        else:
            ph = _address("h", h, shape, _BF16, dev)
    elif h is not None:
        raise ValueError("h needs pre")
    if post is not None:
        w, b = post
        post_w = _vector("post weight", w, C, dev)
        if b is not None:
            post_b = _vector("post bias", b, C, dev)
    _launch((_lib or load()).swin_wattn_block_norm, dev, stream, _plain("x", x, dtype, dev), pf, pre_w, pre_b, post_w, post_b,
            None if gate is None else _vector("gate", gate, C, dev),
            None if keep is None else _vector("keep", keep, samples, dev), py, ph, tokens, C, samples, code,
            _kind_code(kind), alpha, eps)
    return y, h


_NORM_GRADS = ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate")


def block_norm_bwd(y, f=None, dh=None, dy=None, pre=None, post=None, gate=None, keep=None, alpha=1.0, kind="layer",
                   eps=1e-5, dx=None, df=None, grads=None, accumulate=False, workspace=None, stream=None):
    """The gradients of block_norm, for dh (of h, bf16; exactly with pre) and dy (of y's other uses, of
    y's dtype, or None). y is the forward's y (its x, without f); f, pre, post, gate, keep, alpha, kind and
    eps are the forward's. Returns (dx, df, grads): dx of y's dtype (into dx, which may be dy itself),
    df in bf16 or None without f, and a dict of the fp32 gradients of the parameters that are there:
    "pre_weight", "pre_bias", "post_weight", "post_bias", "gate". grads, such a dict: only these are
    computed, written there, or with accumulate added to. workspace: a uint8 tensor of
    swin_wattn_block_norm_bwd_workspace_bytes (allocated here when not given)."""
    dev, shape, dtype = _device_of("y", y), y.shape, y.dtype
    tokens, C, samples = _block_shape(shape, f, post, gate, keep, alpha)
    code = _float_code("y", y)
    if (dh is None) != (pre is None):
        raise ValueError("dh and pre belong together: one of them is None")
    if dh is None and dy is None:
        raise ValueError("neither dh nor dy is given: there is no gradient")
    if f is None and df is not None:
        raise ValueError("df needs f")
    pf = pdh = pdf = pre_w = post_w = post_b = None
    there = []
    if pre is not None:
        w, b = pre
        pre_w, pdh = _vector("pre weight", w, C, dev), _address("dh", dh, shape, _BF16, dev)
        there.append("pre_weight")
        if b is not None:
            there.append("pre_bias")
    if post is not None:
        w, b = post
        post_w = _vector("post weight", w, C, dev)
        there.append("post_weight")
        if b is not None:
            post_b = _vector("post bias", b, C, dev)
            there.append("post_bias")
    if gate is not None:
        there.append("gate")
    if grads is None:
        if accumulate:
            raise ValueError("accumulate needs the grads to add to")
        grads = dict(zip(there, _vectors(len(there), C, dev, stream)))
        pg = [None if (t := grads.get(k)) is None else t.data_ptr() for k in _NORM_GRADS]
    else:
        for k in grads:
            if k not in there:
                raise ValueError(f"grads has {k!r}, which the call has no parameter for")
        pg = [_vector(k, grads[k], C, dev) if k in grads else None for k in _NORM_GRADS]
    if dx is None:
        dx = _empty(shape, dtype, dev, stream)
        pdx = dx.data_ptr()
    else:
        pdx = _address("dx", dx, shape, dtype, dev)
    if f is not None:
        pf = _address("f", f, shape, _BF16, dev)
        if df is None:
            df = _empty(shape, _BF16, dev, stream)
            pdf = df.data_ptr()
        else:
            pdf = _address("df", df, shape, _BF16, dev)
    if workspace is None:
        workspace = _empty((max(swin_wattn_block_norm_bwd_workspace_bytes(tokens, C), 1),), _U8, dev, stream)
    _launch((_lib or load()).swin_wattn_block_norm_bwd, dev, stream, _plain("y", y, dtype, dev), pf, pdh,
            None if dy is None else _address("dy", dy, shape, dtype, dev), pre_w, post_w, post_b,
            None if gate is None else _vector("gate", gate, C, dev),
            None if keep is None else _vector("keep", keep, samples, dev), pdx, pdf, *pg, tokens, C, samples, code,
            _kind_code(kind), alpha, eps, 1 if accumulate else 0, _plain("workspace", workspace, _U8, dev), workspace.numel())
    return dx, df, grads


class GradClip:
    """Clipping by the norm over all gradients of a model: a plan over the fp32 and bf16 CUDA tensors
    `grads` (of any sizes, contiguous), which are checked once and kept. Each call computes
    n = scale |grads| and writes grads * scale * min(1, max_norm / (n + eps)) to `out`, tensors of the
    same shapes and dtypes (the gradients themselves when not given). max_norm is finite; with 3.4e38 and a scale of 1
    a call in place gives the norm alone and leaves finite gradients as they are.

    The plan is of the tensors' memory: it copies a list of it to the device and waits for the stream. It is made once,
    outside of captures, for gradients that stay where they are (written into given tensors, or zeroed in place);
    gradients that are dropped and made anew at each step need a new plan at each step. Its workspace serves one stream
    at a time; a call may bring its own. A captured call reads the plan's list and, without one of its own, its workspace
    on every replay: keep the plan as long as the graph."""

    handle = None

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if not self.grads:
            raise ValueError("grads is empty")
        if len(self.out) != len(self.grads):
            raise ValueError(f"out has {len(self.out)} tensors, grads {len(self.grads)}")
        self.dev = dev = _device_of("grads[0]", self.grads[0])
        codes = [_float_code(f"grads[{i}]", g) for i, g in enumerate(self.grads)]
        ins = [_plain(f"grads[{i}]", g, g.dtype, dev) for i, g in enumerate(self.grads)]
        outs = [_address(f"out[{i}]", o, g.shape, g.dtype, dev) for i, (g, o) in enumerate(zip(self.grads, self.out))]
        sizes = [g.numel() for g in self.grads]
        size = swin_wattn_clip_list_bytes(sizes, codes)
        # the list of the tensors' pieces, then the workspace, of the current stream's memory
        room = _empty((size + swin_wattn_clip_workspace_bytes() + 256,), _U8, dev, None)
        self._home = torch._C._cuda_getCurrentRawStream(dev)
        with torch.cuda.device(dev):
            rc, self.handle = swin_wattn_clip_plan(ins, outs, sizes, codes, room.data_ptr(), size, self._home)
        if rc != OK:
            raise SwinWAttnError("swin_wattn_clip_plan", rc)
        at = (size + 255) & -256
        self._room, self.workspace = room, room[at:at + swin_wattn_clip_workspace_bytes()]

    def __call__(self, max_norm, scale=1.0, eps=1e-6, norm=None, workspace=None, stream=None):
        """Clips; returns the norm n, an fp32 tensor [1] (into norm when given)."""
        dev = self.dev
        if norm is None:
            norm = _empty((1,), _F32, dev, stream)
            pn = norm.data_ptr()
        else:
            pn = _address("norm", norm, (1,), _F32, dev)
        if workspace is None:
            workspace = self.workspace
        if (torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream) != self._home:
            # the list is not given to anyone else while that stream may read it
            self._room.record_stream(torch.cuda.current_stream(dev) if stream is None else stream)
        _launch((_lib or load()).swin_wattn_clip_grad_norm, dev, stream, self.handle, max_norm, scale, eps, pn,
                _plain("workspace", workspace, _U8, dev), workspace.numel())
        return norm

    def close(self):
        if self.handle:
            swin_wattn_clip_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _format_code(format):
    code = FP4_FORMATS.get(format) if type(format) is str else format
    if code is None or not NVFP4 <= code <= MXFP4:
        raise ValueError(f"unknown format {format!r}: one of {sorted(FP4_FORMATS)} or NVFP4, MXFP4")
    return code


def _fp4_sizes(shape, fmt):
    """Rows, K and the bytes of the scales of a matrix [..., K]."""
    if not shape:
        raise ValueError("the matrix has no dimensions")
    K = shape[-1]
    rows = shape[0] if len(shape) == 2 else shape[:-1].numel()
    if rows > _INT_MAX or K > _INT_MAX:
        raise _too_large(rows, K)
    return rows, K, (rows + 127) // 128 * ((K // (32 if fmt else 16) + 3) // 4) * 512


class Fp4Tensor:
    """A matrix [..., K] in microscaled 4-bit floating point: `codes`, a uint8 tensor [..., K / 2]; `scales`,
    a flat uint8 tensor in the tensor core's tiles; `tensor_scale`, fp32 [1], of NVFP4 (else None);
    `format`, NVFP4 or MXFP4; `shape`, of the matrix. The tensors are checked here, once."""

    __slots__ = ("_data", "_parts", "_at", "_dev", "_rows", "_K", "format", "shape")

    def __init__(self, codes, scales, tensor_scale, format, shape):
        self.format, self.shape = fmt, shape = _format_code(format), torch.Size(shape)
        self._rows, self._K, size = _fp4_sizes(shape, fmt)
        self._dev = dev = _device_of("codes", codes)
        if (tensor_scale is None) != (fmt == MXFP4):
            raise ValueError("NVFP4 has a scale of the tensor, MXFP4 has none")
        self._data, self._parts = None, (codes, scales, tensor_scale)
        self._at = (_address("codes", codes, (*shape[:-1], self._K // 2), _U8, dev), _address("scales", scales, (size,), _U8, dev),
                    None if tensor_scale is None else _address("tensor_scale", tensor_scale, (1,), _F32, dev))

    @classmethod
    def _empty(cls, shape, fmt, scale, dev, stream):
        """Room for a matrix, in one allocation: codes, scales, the tensor's scale (unless `scale` is it) and what
        finding it takes, each from a multiple of 256 bytes on."""
        self = cls.__new__(cls)
        self.format, self.shape, self._dev = fmt, shape, dev
        self._rows, self._K, size = _fp4_sizes(shape, fmt)
        codes = (self._rows * (self._K // 2) + 255) & -256
        own = fmt == NVFP4 and scale is None
        self._data = data = _empty((codes + size + (256 + _fp4_scratch() if own else 0),), _U8, dev, stream)
        p = data.data_ptr()
        self._parts = scale
        self._at = (p, p + codes, p + codes + size if own else None if scale is None else
                    _address("scale", scale, (1,), _F32, dev))
        return self

    @property
    def codes(self):
        if self._data is None:
            return self._parts[0]
        return self._data[:self._rows * (self._K // 2)].view(*self.shape[:-1], self._K // 2)

    @property
    def scales(self):
        if self._data is None:
            return self._parts[1]
        at = self._at[1] - self._at[0]
        return self._data[at:at + _fp4_sizes(self.shape, self.format)[2]]

    @property
    def tensor_scale(self):
        if self._data is None:
            return self._parts[2]
        if self._parts is not None or self.format == MXFP4:
            return self._parts  # the given scale, or none
        at = self._at[2] - self._at[0]
        return self._data[at:at + 4].view(_F32)


_scratch_bytes = None


def _fp4_scratch():
    global _scratch_bytes
    if _scratch_bytes is None:
        _scratch_bytes = swin_wattn_fp4_workspace_bytes()
    return _scratch_bytes


def quantize_fp4(x, format="nvfp4", scale=None, out=None, workspace=None, stream=None):
    """The bf16 or fp32 CUDA tensor x [..., K] in microscaled 4-bit floating point, an Fp4Tensor (`out` when given):
    "nvfp4", blocks of 16 with E4M3 scales and a scale of the tensor, or "mxfp4", blocks of 32 with powers
    of two. scale, fp32 [1], is the tensor's scale of NVFP4, calibrated ahead of time; without it it is taken
    from x and written to out's. workspace: a uint8 tensor of swin_wattn_fp4_workspace_bytes (part of the result when not given)."""
    dev, shape, fmt, code = _device_of("x", x), x.shape, _format_code(format), _float_code("x", x)
    if fmt == MXFP4 and scale is not None:
        raise ValueError("MXFP4 has no scale of the tensor")
    own = fmt == NVFP4 and scale is None
    if out is None:
        out = Fp4Tensor._empty(shape, fmt, scale, dev, stream)
    elif out.format != fmt or out.shape != shape:
        raise ValueError(f"out is of format {out.format} and shape {tuple(out.shape)}, not {fmt} and {tuple(shape)}")
    elif out._dev != dev:
        raise ValueError(f"out is on cuda:{out._dev}, not on cuda:{dev}")
    elif scale is not None and out.tensor_scale.data_ptr() != scale.data_ptr():
        raise ValueError("out.tensor_scale is not the given scale")
    elif own and out._data is not None and out._parts is not None:
        raise ValueError("out was made with a given scale: pass it again (it is not overwritten)")
    ws, size = None, 0
    if own:
        if workspace is None and out._data is not None and out._parts is None:
            ws, size = out._at[2] + 256, _fp4_scratch()
        else:
            if workspace is None:
                workspace = _empty((_fp4_scratch(),), _U8, dev, stream)
            ws, size = _plain("workspace", workspace, _U8, dev), workspace.numel()
    _launch((_lib or load()).swin_wattn_fp4_quantize, dev, stream, _plain("x", x, x.dtype, dev), *out._at, out._rows, out._K,
            fmt, code, 0 if own else 1, ws, size)
    return out


def dequantize_fp4(q, dtype=torch.bfloat16, out=None, stream=None):
    """The values that an Fp4Tensor stands for, in bf16 or fp32 (into `out` when given)."""
    dev = q._dev
    if out is None:
        out = _empty(q.shape, dtype, dev, stream)
        po = out.data_ptr()
    else:
        po = _address("out", out, q.shape, out.dtype, dev)
    _launch((_lib or load()).swin_wattn_fp4_dequantize, dev, stream, *q._at, po, q._rows, q._K, q.format,
            _float_code("out", out))
    return out


def linear_fp4(x, w, b=None, act=ACT_NONE, residual=None, x_scale=None, y=None, workspace=None, status=None, stream=None):
    """residual + act(x W^T + b) on 4-bit operands: w [N, K] an Fp4Tensor (a weight quantised once), x [..., K] an
    Fp4Tensor of the same format, or a bf16 or fp32 CUDA tensor, which is quantised on the way (x_scale: its tensor's
    scale for NVFP4, fp32 [1], else taken from x; workspace: a uint8 tensor of swin_wattn_linear_fp4_workspace_bytes,
    allocated here when needed and not given). The rest as for linear; y is bf16 [..., N]."""
    dev, ws, xs, fmt = w._dev, w.shape, x.shape, w.format
    if len(ws) != 2 or not xs or xs[-1] != ws[1]:
        raise ValueError(f"x and w have shapes {tuple(xs)} and {tuple(ws)}: not [..., K] and [N, K]")
    N, K = ws
    tokens, shape = _leading(xs, N)
    if y is None:
        y = _empty(shape, _BF16, dev, stream)
        py = y.data_ptr()
    else:
        py = _address("y", y, shape, _BF16, dev)
    rest = (None if b is None else _vector("b", b, N, dev),
            None if residual is None else _address("residual", residual, shape, _BF16, dev), py, tokens, K, N, fmt)
    if isinstance(x, Fp4Tensor):
        if x_scale is not None:
            raise ValueError("x is quantised: it has its own scale")
        if x.format != fmt:
            raise ValueError(f"x and w have the formats {x.format} and {fmt}")
        if x._dev != dev:
            raise ValueError(f"x is on cuda:{x._dev}, not on cuda:{dev}")
        _call((_lib or load()).swin_wattn_linear_fp4, dev, stream, status, *x._at, *w._at, *rest, _act_code(act))
        return y
    code = _float_code("x", x)
    if tokens > _INT_MAX:
        raise _too_large(tokens)
    if x_scale is not None and fmt == MXFP4:
        raise ValueError("MXFP4 has no scale of the tensor")
    if workspace is not None:
        pw, size = _plain("workspace", workspace, _U8, dev), workspace.numel()
    elif size := (_lib or load()).swin_wattn_linear_fp4_workspace_bytes(tokens, K, N, fmt, x_scale is not None):
        workspace = _empty((size,), _U8, dev, stream)
        pw = workspace.data_ptr()
    else:
        pw = None
    _call((_lib or load()).swin_wattn_linear_fp4_of, dev, stream, status, _plain("x", x, x.dtype, dev),
          None if x_scale is None else _vector("x_scale", x_scale, 1, dev), *w._at, *rest, code, _act_code(act), pw, size)
    return y


def swin_wattn_fwd_fp8(plan, qkv8_ptr, scale_q, scale_k, scale_v, out_ptr, stream):
    return load().swin_wattn_fwd_fp8(plan, qkv8_ptr, scale_q, scale_k, scale_v, out_ptr, stream)


def swin_wattn_set_fwd_kernel(plan, kernel):
    return load().swin_wattn_set_fwd_kernel(plan, kernel)


def swin_wattn_fwd_kernel(plan):
    return load().swin_wattn_fwd_kernel(plan)


def swin_wattn_set_bwd_kernel(plan, kernel):
    return load().swin_wattn_set_bwd_kernel(plan, kernel)


def swin_wattn_bwd_kernel(plan):
    return load().swin_wattn_bwd_kernel(plan)


def swin_wattn_device_status(plan, stream):
    return load().swin_wattn_device_status(plan, stream)


def swin_wattn_destroy(plan):
    return load().swin_wattn_destroy(plan)


def swin_wattn_status_string(status):
    return load().swin_wattn_status_string(status).decode()


def swin_wattn_last_error():
    return load().swin_wattn_last_error().decode()


def swin_wattn_launch_count(reset=False):
    return int(load().swin_wattn_launch_count(1 if reset else 0))


# ---- torch convenience wrapper ---------------------------------------------------------

def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


class WindowAttention:
    """A plan for one layer shape, driven with torch CUDA tensors.

    ``table`` is the fp32 [(2M-1)^2, nH] bias table on the GPU. Activations are bf16 or
    fp32 [B,H,W,3C] tensors (contiguous); outputs are allocated by the caller or here.
    """

    def __init__(self, B, H, W, C, num_heads, window, shift, table, dtype="bf16", stream=None):
        import torch
        self.B, self.H, self.W, self.C = B, H, W, C
        self.nH, self.M, self.s = num_heads, window, shift
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        code = BF16 if dtype == "bf16" else FP32
        rc, h = swin_wattn_plan(B, H, W, C, num_heads, window, shift, code, table.data_ptr(),
                                _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_plan", rc)
        self.handle = h

    def set_fwd_kernel(self, kernel):
        """KERNEL_AUTO, KERNEL_MMA_SYNC or KERNEL_TCGEN05 for later forwards."""
        rc = swin_wattn_set_fwd_kernel(self.handle, kernel)
        if rc != OK:
            raise SwinWAttnError("swin_wattn_set_fwd_kernel", rc)

    @property
    def fwd_kernel(self):
        return swin_wattn_fwd_kernel(self.handle)

    def set_bwd_kernel(self, kernel):
        """KERNEL_AUTO, KERNEL_MMA_SYNC or KERNEL_TCGEN05 for later backwards."""
        rc = swin_wattn_set_bwd_kernel(self.handle, kernel)
        if rc != OK:
            raise SwinWAttnError("swin_wattn_set_bwd_kernel", rc)

    @property
    def bwd_kernel(self):
        return swin_wattn_bwd_kernel(self.handle)

    def device_status(self, stream=None):
        """Synchronise and raise if a bounded device wait ran out since the last check."""
        rc = swin_wattn_device_status(self.handle, _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_device_status", rc)

    def set_bias(self, table, stream=None):
        rc = swin_wattn_set_bias(self.handle, table.data_ptr(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_set_bias", rc)

    def fwd(self, qkv, out=None, stream=None):
        import torch
        if out is None:
            out = torch.empty(self.B, self.H, self.W, self.C, dtype=self.dtype, device=qkv.device)
        rc = swin_wattn_fwd(self.handle, qkv.data_ptr(), out.data_ptr(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_fwd", rc)
        return out

    def fwd_fp8(self, qkv8, scales, out=None, stream=None):
        """Forward on 8-bit operands: qkv8 a [B,H,W,3C] CUDA tensor of OCP FP8 E4M3 bytes
        (torch.float8_e4m3fn or uint8), scales (scale_q, scale_k, scale_v); bf16 output."""
        import torch
        if out is None:
            out = torch.empty(self.B, self.H, self.W, self.C, dtype=torch.bfloat16, device=qkv8.device)
        sq, sk, sv = (float(x) for x in scales)
        rc = swin_wattn_fwd_fp8(self.handle, qkv8.data_ptr(), sq, sk, sv, out.data_ptr(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_fwd_fp8", rc)
        return out

    def fwd_host(self, qkv_host, out_host, dev_qkv, dev_out, stream=None):
        """Host-resident qkv -> host-resident out through the library's host entry point
        (copies and kernel in order on the stream; synchronise before reading out_host)."""
        rc = swin_wattn_fwd_host(self.handle, qkv_host.data_ptr(), out_host.data_ptr(),
                                 dev_qkv.data_ptr(), dev_out.data_ptr(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_fwd_host", rc)
        return out_host

    def bwd(self, qkv, dout, dqkv=None, dtable=None, stream=None):
        import torch
        if dqkv is None:
            dqkv = torch.empty_like(qkv)
        if dtable is None:
            dtable = torch.empty((2 * self.M - 1) ** 2, self.nH, dtype=torch.float32,
                                 device=qkv.device)
        rc = swin_wattn_bwd(self.handle, qkv.data_ptr(), dout.data_ptr(), dqkv.data_ptr(),
                            dtable.data_ptr(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_bwd", rc)
        return dqkv, dtable

    def debug_maps(self, stream=None):
        import torch
        dev = torch.device("cuda")
        N, nW = self.M * self.M, (self.H // self.M) * (self.W // self.M)
        gather = torch.empty(nW, N, dtype=torch.int32, device=dev)
        relidx = torch.empty(N, N, dtype=torch.int32, device=dev)
        mask = torch.empty(nW, N, N, dtype=torch.float32, device=dev)
        dense = torch.empty(self.nH, N, N, dtype=torch.float32, device=dev)
        rc = swin_wattn_debug_maps(self.handle, gather.data_ptr(), relidx.data_ptr(),
                                   mask.data_ptr(), dense.data_ptr(), _stream_handle(stream))
        if rc != OK:
            raise SwinWAttnError("swin_wattn_debug_maps", rc)
        return gather, relidx, mask, dense

    def close(self):
        if getattr(self, "handle", None):
            swin_wattn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
