/*
 * swin_wattn: fused Swin window / shifted-window multi-head attention (W-MSA / SW-MSA)
 * on one NVIDIA GB300 GPU (sm_103a). C ABI; every call is asynchronous on the stream
 * it is given and reports failure only through its return code.
 *
 * What is computed (sources cited by page and section):
 *  - NVIDIA "visual large-model training and inference optimisation" talk, full
 *    transcript (uticex.com, article 1598), section 1: attention among the tokens of each
 *    non-overlapping M x M window, a cyclic window shift that bridges window borders, and
 *    a learned relative position bias added to the attention logits.
 *  - same transcript, section 2: shift, window partition and window reverse are index
 *    mappings only; the mask and the bias reach the fused attention as tensors.
 *  - same transcript, section 3: the relative-position bias lookup runs once, as
 *    preprocessing, producing a dense per-head bias; batch GEMM + softmax + batch GEMM
 *    run as one fused kernel whose loads and stores absorb the layout transposes.
 *  - Baidu AIAK-Training talk (jxzklqfsx.com, article 743345), section 2, the fused
 *    WindowAttention case: one kernel staging HBM -> shared memory -> registers, tensor
 *    cores for both products, and a backward that recomputes instead of reloading.
 *
 * For an activation qkv of shape [B, H, W, 3C] (channel t*C + h*hd + d, t in {q,k,v},
 * head h < nH, hd = C/nH = 32), window size M and shift s (0 <= s < M):
 *   rolled token (y, x) reads original token ((y+s) mod H, (x+s) mod W);
 *   windows are row-major over (H/M, W/M), tokens row-major inside a window;
 *   logit(i,j) = hd^-0.5 * q_i.k_j + table[idx(i,j), h] + mask_w(i,j), with
 *   idx(i,j) = (yi-yj+M-1)*(2M-1) + (xi-xj+M-1) for local window positions,
 *   mask_w(i,j) = -100 when the two tokens carry different shift-region labels
 *   (per axis of length L on the rolled grid: [0,L-M), [L-M,L-s), [L-s,L); label =
 *   3*region_y + region_x), else 0; no mask when s = 0;
 *   P = row softmax of the logits, O = P V, written to channel h*hd + d of the same
 *   token position it was read from: out has shape [B, H, W, C].
 *
 * Conventions for every entry point:
 *  - Tensor pointers are device pointers (cudaMalloc, or torch CUDA tensors), contiguous
 *    in the layouts above, 16-byte aligned, owned by the caller. A host pointer is
 *    rejected with SWIN_WATTN_ERR_INVALID_ARG before any launch.
 *  - Activation dtype is fixed per plan: SWIN_WATTN_BF16 (bf16 in and out) or
 *    SWIN_WATTN_FP32 (fp32 in and out; values are rounded to bf16, round-to-nearest-
 *    even, on load). Arithmetic: bf16 tensor-core products with fp32 accumulation,
 *    fp32 softmax.
 *  - The bias table is fp32 [(2M-1)^2, nH], row-major; its gradient likewise.
 *  - Errors come back as status codes; nothing aborts, traps or throws across the ABI.
 *    After SWIN_WATTN_ERR_CUDA, swin_wattn_last_error() holds the CUDA error text of the
 *    calling thread.
 */
#ifndef SWIN_WATTN_H
#define SWIN_WATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t */

typedef struct swin_wattn_plan_s* swin_wattn_plan_t;

enum swin_wattn_status {
  SWIN_WATTN_OK = 0,
  SWIN_WATTN_ERR_INVALID_ARG = 1,  /* null/host pointer, bad dtype, s out of range, ... */
  SWIN_WATTN_ERR_UNSUPPORTED = 2,  /* M not in {4,7,12}, head width != 32, H%M or W%M != 0 */
  SWIN_WATTN_ERR_MISALIGNED = 3,   /* tensor pointer not 16-byte aligned (table: 4-byte) */
  SWIN_WATTN_ERR_BAD_PLAN = 4,     /* null, destroyed or foreign plan handle */
  SWIN_WATTN_ERR_CUDA = 5,         /* a CUDA runtime call failed; see swin_wattn_last_error */
  SWIN_WATTN_ERR_TIMEOUT = 6       /* a bounded device-side wait ran out (see
                                      swin_wattn_device_status) */
};

enum swin_wattn_dtype { SWIN_WATTN_BF16 = 0, SWIN_WATTN_FP32 = 1 };

/* Forward and backward kernels (swin_wattn_set_fwd_kernel, swin_wattn_set_bwd_kernel). */
enum swin_wattn_kernel {
  SWIN_WATTN_KERNEL_AUTO = 0,      /* the faster kernel as measured (see the setters below) */
  SWIN_WATTN_KERNEL_MMA_SYNC = 1,  /* warp-level mma.sync kernel: every M, both dtypes */
  SWIN_WATTN_KERNEL_TCGEN05 = 2    /* tensor-memory kernels: M = 7 or 12 with bf16 */
};

/* Activations of the MLP's products (swin_wattn_linear, swin_wattn_linear_bwd_data). */
enum swin_wattn_activation {
  SWIN_WATTN_ACT_NONE = 0,
  SWIN_WATTN_ACT_RELU = 1,      /* max(z, 0); derivative 0 at z = 0 */
  SWIN_WATTN_ACT_GELU = 2,      /* z Phi(z), Phi the normal distribution function */
  SWIN_WATTN_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
  SWIN_WATTN_ACT_SILU = 4       /* z / (1 + exp(-z)) */
};

/* Norms of swin_wattn_block_norm, and formats of the 4-bit operands. */
enum swin_wattn_norm {
  SWIN_WATTN_NORM_LAYER = 0, /* (v - mean) / sqrt(var + eps) */
  SWIN_WATTN_NORM_RMS = 1    /* v / sqrt(mean of v^2 + eps) */
};
enum swin_wattn_fp4_format {
  SWIN_WATTN_NVFP4 = 0, /* blocks of 16 with an E4M3 scale, and one fp32 scale of the tensor */
  SWIN_WATTN_MXFP4 = 1  /* blocks of 32 with a power of two (E8M0) */
};

/*
 * Create a plan for one layer shape and run the preprocessing on `stream`:
 * the dense bias [nH, M^2, M^2] is expanded from `bias_table` (the lookup done once, as
 * in section 3 of the NVIDIA transcript) and, for s > 0, the shift mask [nW, M^2, M^2]
 * (nW = (H/M)(W/M), values 0 / -100) is built.
 *   out         receives the plan handle (set to NULL on failure).
 *   B           batch (B = 0 is allowed: every call on the plan is then a no-op,
 *               except that swin_wattn_bwd still zeroes dtable).
 *   H, W        token grid; multiples of M.
 *   C           channels per q/k/v; C = 32 * num_heads.
 *   window      M in {4, 7, 12}.  shift: s in [0, M).
 *   dtype       SWIN_WATTN_BF16 or SWIN_WATTN_FP32 activation I/O.
 *   bias_table  device fp32 [(2M-1)^2, num_heads]; read during this call's launch only.
 * The plan owns its dense bias, its mask and the backward's reduction scratch (device
 * memory allocated here, freed by swin_wattn_destroy). A plan is used by one stream at a
 * time; swin_wattn_fwd and swin_wattn_bwd allocate nothing.
 */
int swin_wattn_plan(swin_wattn_plan_t* out, int B, int H, int W, int C, int num_heads,
                    int window, int shift, int dtype, const float* bias_table,
                    struct CUstream_st* stream);

/* Re-expand the dense bias from an updated table (training). Same table layout. */
int swin_wattn_set_bias(swin_wattn_plan_t plan, const float* bias_table,
                        struct CUstream_st* stream);

/*
 * Forward: qkv [B,H,W,3C] -> out [B,H,W,C] (plan dtype). One kernel launch: the roll and
 * window partition are folded into the load addressing and the reverse and un-roll into
 * the store; logits, bias, mask and softmax stay on chip. `out` must not overlap `qkv`.
 */
int swin_wattn_fwd(swin_wattn_plan_t plan, const void* qkv, void* out,
                   struct CUstream_st* stream);

/*
 * Forward on host-resident activations, for callers whose data lives in host memory:
 * copies qkv_host [B,H,W,3C] into the caller-owned device buffer dev_qkv, runs the same
 * kernel as swin_wattn_fwd into dev_out, and copies dev_out back to out_host [B,H,W,C].
 * The batch is cut into up to four chunks that flow through a copy-in queue, `stream`
 * (the kernels) and a copy-out queue, so both copy directions and the compute overlap;
 * `stream` waits for the last copy-out, so the whole call is ordered on `stream`
 * (synchronise it before reading out_host). The two copy queues and their events are
 * created by the plan's first call. Host buffers should be page-locked (cudaHostAlloc,
 * or torch pin_memory) for the copies to be asynchronous. dev_qkv and dev_out must be
 * device pointers (16-byte aligned).
 */
int swin_wattn_fwd_host(swin_wattn_plan_t plan, const void* qkv_host, void* out_host,
                        void* dev_qkv, void* dev_out, struct CUstream_st* stream);

/*
 * Backward for an upstream gradient dout [B,H,W,C] (plan dtype):
 *   dqkv   [B,H,W,3C] plan dtype, fully overwritten (dq, dk, dv at the channels the
 *          forward read q, k, v from);
 *   dtable [(2M-1)^2, nH] fp32, overwritten (not accumulated) with the bias-table
 *          gradient summed over every batch, window and (i, j) pair.
 * The forward's probabilities are recomputed, not stored (AIAK-Training talk,
 * section 2). Deterministic: the same inputs give bit-identical outputs.
 */
int swin_wattn_bwd(swin_wattn_plan_t plan, const void* qkv, const void* dout, void* dqkv,
                   float* dtable, struct CUstream_st* stream);

/*
 * Backward without any device allocation (the pages have no counterpart: this entry
 * point exists for callers that cannot allocate device memory when they run the
 * backward, e.g. runtimes that fix their device memory plan at start-up and forbid any
 * later cudaMalloc, or frameworks whose own allocator must own every device byte; such
 * callers cannot create a plan, because a plan allocates).
 *
 * Same arguments and results as swin_wattn_plan followed by swin_wattn_bwd with the
 * MMA_SYNC backward kernel (qkv, dout, dqkv, dtable and the bias table are the caller's
 * device buffers; window must be 4 or 7), but no plan is made and nothing is allocated or
 * freed: the working memory (bias
 * fragments, mask bits, per-CTA table-gradient partials) lives in one fixed 2 MiB
 * device array inside the library, which every GPU that loads the library holds until
 * the process exits. A shape whose working memory exceeds 2 MiB is refused with
 * SWIN_WATTN_ERR_UNSUPPORTED and the reason in swin_wattn_last_error().
 *
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress)
 * with that device current; make that first call before any stream capture. The address
 * is kept for the life of the process, so do not call this entry point on a device after
 * a cudaDeviceReset of that device (the reset unloads the array it points into). Every
 * call on a device shares the one array and rewrites the parts it reads before reading
 * them, so two calls that overlap on the GPU (different streams without ordering between
 * them) race: order them. Three kernel launches on `stream` (fragments, backward,
 * table-gradient sum), counted by swin_wattn_launch_count.
 */
int swin_wattn_bwd_noalloc(const void* qkv, const void* dout, void* dqkv, float* dtable,
                           const float* bias_table, int B, int H, int W, int C, int num_heads,
                           int window, int shift, int dtype, struct CUstream_st* stream);

/*
 * Debug dumps of the plan's index maps and preprocessed tensors (device pointers, any
 * may be NULL to skip):
 *   gather     int32 [nW, M^2]: original token index y*W + x that window w, slot i
 *              reads (and writes), computed by the same addressing as the kernels;
 *   relidx     int32 [M^2, M^2]: relative position index idx(i, j);
 *   mask       fp32 [nW, M^2, M^2]: the plan's shift mask (all zeros when s = 0);
 *   dense_bias fp32 [nH, M^2, M^2]: the plan's expanded bias.
 */
int swin_wattn_debug_maps(swin_wattn_plan_t plan, int32_t* gather, int32_t* relidx,
                          float* mask, float* dense_bias, struct CUstream_st* stream);

/*
 * The producer step in front of the attention (NVIDIA talk, section 2, lists LayerNorm and
 * the qkv GEMM among the operations fused around the window attention): for each of
 * `tokens` tokens,
 *   xn = (x - mean) / sqrt(var + eps) * gamma + beta   (mean, population variance over C)
 *   qkv = xn W^T + b
 *   x      bf16 [tokens, C] (e.g. a [B,H,W,C] activation), device, 16-byte aligned;
 *   gamma, beta fp32 [C]; b fp32 [3C]; device;
 *   w_qkv  bf16 [3C, C] (row n = output channel n, in the order q | k | v, head-major);
 *   qkv    bf16 [tokens, 3C], device, 16-byte aligned, written (the attention's input);
 *   workspace  caller-owned device memory of at least swin_wattn_qkv_workspace_bytes(C,
 *          tokens) bytes, 256-byte aligned, overwritten (the gamma-folded weights, two
 *          per-channel vectors and the per-token statistics); one call at a time per
 *          workspace;
 *   status optional device int (may be NULL): bit 0 is OR-ed in if a bounded device wait
 *          ran out (then qkv is not valid).
 * The normalisation is applied on the other side of the product:
 *   xn W^T + b = rstd (x W'^T) - rstd mean u + v,  W' = bf16(gamma * W) (per input channel),
 *   u = row sums of W', v = beta W^T + b,
 * with the row statistics in fp32 and the product accumulated in fp32 on bf16 x and W';
 * qkv is rounded to bf16. C must be a multiple of 32 in [32, 1536]. The cyclic shift and
 * window partition are not applied here: the attention folds them into its loads. Two
 * kernel launches on `stream` (the weight fold, with the token statistics when the product
 * does not sum them itself; the product); nothing is allocated.
 * swin_wattn_qkv_workspace_bytes returns 0 for an unsupported C.
 */
size_t swin_wattn_qkv_workspace_bytes(int C, int tokens);
int swin_wattn_qkv_proj(const void* x, const float* gamma, const float* beta, const void* w_qkv,
                        const float* b_qkv, void* qkv, int tokens, int C, float eps, void* workspace,
                        size_t workspace_bytes, int* status, struct CUstream_st* stream);

/*
 * The producer step with its weights prepared once (NVIDIA Swin talk, section 3: inference
 * may transform the qkv weight and bias ahead of time). swin_wattn_qkv_prepare writes W',
 * u and v (as above) for gamma, beta, w_qkv, b_qkv into `prepared` (device, 256-byte
 * aligned, at least swin_wattn_qkv_prepared_bytes(C) bytes; one launch). Then each
 * swin_wattn_qkv_proj_prepared call computes qkv for x from them, with the same arithmetic
 * and results as swin_wattn_qkv_proj; it reads `prepared` and uses `stats_workspace`
 * (device, 16-byte aligned, at least swin_wattn_qkv_stats_bytes(tokens) bytes,
 * overwritten; one call at a time per workspace) for the per-token statistics. One or two
 * launches (the statistics pass where the product does not sum them itself; the product).
 * Errors as for swin_wattn_qkv_proj. The size queries return 0 for unsupported arguments.
 */
size_t swin_wattn_qkv_prepared_bytes(int C);
size_t swin_wattn_qkv_stats_bytes(int tokens);
int swin_wattn_qkv_prepare(const float* gamma, const float* beta, const void* w_qkv, const float* b_qkv, int C,
                           void* prepared, size_t prepared_bytes, struct CUstream_st* stream);
int swin_wattn_qkv_proj_prepared(const void* x, const void* prepared, void* qkv, int tokens, int C, float eps,
                                 void* stats_workspace, size_t stats_bytes, int* status,
                                 struct CUstream_st* stream);

/*
 * The producer step on prepared weights with OCP FP8 E4M3 output, the input of
 * swin_wattn_fwd_fp8 (NVIDIA Swin talk, section 3: the inference path takes its GEMMs to 8
 * bits with scales calibrated ahead of time; here the qkv the attention reads): the same
 * qkv as swin_wattn_qkv_proj_prepared, in fp32, then for each channel of tensor t (q, k, v)
 *   qkv8 = E4M3(qkv / scale_t), rounded to nearest even, saturated to +-448;
 *   qkv8   device, 16-byte aligned: [tokens, 3C] bytes, written (the token layout of qkv);
 *   scale_q, scale_k, scale_v  one fp32 scale per tensor, finite and positive (static
 *          scaling: e.g. the calibrated max |qkv_t| / 448);
 *   amax   optional device float[3] (may be NULL): max |qkv_t| of this call's fp32 values is
 *          max-ed into amax[t] atomically (the caller zeroes it; a later call can take its
 *          scales from it: delayed scaling).
 * Other arguments and errors as for swin_wattn_qkv_proj_prepared (INVALID_ARG also for a bad
 * scale). One or two launches; nothing is allocated.
 */
int swin_wattn_qkv_proj_prepared_fp8(const void* x, const void* prepared, void* qkv8, int tokens, int C, float eps,
                                     float scale_q, float scale_k, float scale_v, float* amax, void* stats_workspace,
                                     size_t stats_bytes, int* status, struct CUstream_st* stream);

/*
 * The consumer step after the attention: the output projection, then its bias and the
 * residual added, fused into the product's epilogue (NVIDIA Swin talk, uticex.com article
 * 1598, section 3 "inference optimisation": the bias-plus-residual pass in its half2
 * example):
 *   y[t] = residual[t] + o[t] Wp^T + bp   for each token t < tokens.
 * Arguments (device pointers unless stated):
 *   o        bf16 [tokens, C], 16-byte aligned: the attention output (swin_wattn_fwd's
 *            out, channel order h*32 + d);
 *   w_proj   bf16 [C, C] (row n = output channel n);
 *   b_proj   fp32 [C];
 *   residual bf16 [tokens, C], 16-byte aligned: the block input (the shortcut);
 *   y        bf16 [tokens, C], 16-byte aligned, written. y may be the residual buffer
 *            itself (each element is read before it is written) but must not overlap o;
 *   status   optional device int (may be NULL): bit 0 is OR-ed in if a bounded device
 *            wait ran out (then y is not valid).
 * The product is accumulated in fp32 on the bf16 operands, bp and the residual are added
 * in fp32, and y is rounded to bf16. C must be a multiple of 32 in [32, 1536]. One kernel
 * launch on `stream`; nothing is allocated. Errors: INVALID_ARG for negative tokens,
 * overlapping o and y, or a pointer that is not device memory; MISALIGNED for a pointer
 * off its alignment; UNSUPPORTED for C.
 * swin_wattn_linear(o, w_proj, b_proj, residual, y, NULL, tokens, C, C, SWIN_WATTN_ACT_NONE, ...)
 * computes the same, for any C that is a multiple of 8, and is the one to call in new code: it takes
 * as long or less (49 x 768 6.2 against 9.3 us, 3136 x 768 8.6 against 10.3, 50176 x 192 14.5
 * against 14.4). This one stays for its callers.
 */
int swin_wattn_proj_residual(const void* o, const void* w_proj, const float* b_proj, const void* residual,
                             void* y, int tokens, int C, int* status, struct CUstream_st* stream);

/*
 * A product with bias, activation and residual in its epilogue, the two halves of a block's
 * MLP (NVIDIA Swin talk, section 1: a block's FFN; section 3: bias, activation and residual
 * fused into the products around them) and any other dense layer:
 *   z = x W^T + b,   y = residual + act(z)
 * Arguments (device pointers of the current device, contiguous, 16-byte aligned unless
 * stated):
 *   x        bf16 [tokens, K];
 *   w        bf16 [N, K] (row n = output channel n);
 *   b        fp32 [N], 4-byte aligned, or NULL for no bias;
 *   residual bf16 [tokens, N], or NULL for none;
 *   y        bf16 [tokens, N], written. y may be the residual buffer itself (each element is
 *            read before it is written) but must not overlap x, w, or pre;
 *   pre      bf16 [tokens, N], or NULL: z is also written there, rounded to bf16, for
 *            swin_wattn_linear_bwd_data. act is applied to the unrounded z;
 *   tokens   in [0, 2147482624] (0: nothing is done); K, N: multiples of 8 in [8, 32768];
 *   act      SWIN_WATTN_ACT_*;
 *   status   optional device int (may be NULL): bit 0 is OR-ed in if a bounded device wait
 *            ran out (then the results are not valid).
 * The product is accumulated in fp32 on the bf16 operands; bias, activation and residual are
 * applied in fp32 and each result is rounded once. Activations are a fit or hardware exponentials
 * in fp32: GELU is off by at most 7e-6, and by 5e-5 of itself for z < 0 down to -6, the others by
 * 2e-6; NaN gives NaN, +inf gives +inf, -inf gives 0. One kernel launch on `stream`; nothing is
 * allocated. Deterministic. Errors: INVALID_ARG for negative tokens, an unknown act, overlapping
 * buffers, or a pointer that the current device cannot address as its own (another device's
 * memory, host memory that is not mapped); MISALIGNED for a pointer off its alignment;
 * UNSUPPORTED for K, N or tokens out of range.
 */
int swin_wattn_linear(const void* x, const void* w, const float* b, const void* residual, void* y, void* pre,
                      int tokens, int K, int N, int act, int* status, struct CUstream_st* stream);

/*
 * The gradient of a product's input, taken through the activation that made that input:
 *   dx = (dy W) * act'(pre)
 *   dy   bf16 [tokens, N];   w  bf16 [N, K] (the forward's weight);
 *   pre  bf16 [tokens, K], the pre-activation kept by the forward that made x; NULL (and not
 *        read) when act is SWIN_WATTN_ACT_NONE;
 *   dx   bf16 [tokens, K], written. dx may be the pre buffer itself but must not overlap dy
 *        or w.
 * With act NONE, dx = dy W is the gradient of x; with an activation, of the pre-activation
 * that x = act(pre) came from. act' is off by at most 3e-5 for GELU, which shows beside the rounding
 * to bf16 only where act' is near zero (z = -0.75), and by 4e-6 for the others; ReLU's is 0 at 0 and
 * at NaN. Sizes, status, arithmetic and errors as for swin_wattn_linear.
 * One launch.
 */
int swin_wattn_linear_bwd_data(const void* dy, const void* w, const void* pre, void* dx, int tokens, int K, int N,
                               int act, int* status, struct CUstream_st* stream);

/*
 * The gradients of a product's weight and bias:
 *   dw = [dw +] dy^T x,   db = [db +] sum of dy over the tokens
 *   dy   bf16 [tokens, N];   x  bf16 [tokens, K];
 *   dw   [N, K], fp32 or bf16 by `dtype` (SWIN_WATTN_FP32 or SWIN_WATTN_BF16), written;
 *   db   fp32 [N], 4-byte aligned, or NULL;
 *   accumulate  nonzero: the gradients are added to what dw and db hold (in fp32, rounded
 *        once), for several micro-batches; zero: they are overwritten. With no tokens the sum
 *        is empty: dw and db are zeroed, or left as they are when accumulating;
 *   workspace   caller-owned device memory of at least
 *        swin_wattn_linear_bwd_weight_workspace_bytes(tokens, K, N) bytes, 256-byte aligned,
 *        overwritten (partial results of groups of tokens); one call at a time per workspace,
 *        and none of the other buffers.
 * Summed in fp32, in an order that depends on the sizes alone: deterministic. (512 tokens at a time
 * by the tensor cores, whose additions truncate, these rounded to nearest: fp32 results are off by
 * 5e-7 of random sums, relative 2-norm, and by up to 2e-6 where all terms have one sign.) One or two
 * launches; nothing is allocated. dw, db and workspace must not overlap the inputs or one
 * another. Sizes, status and errors as for swin_wattn_linear (INVALID_ARG also for a small
 * workspace or an unknown dtype). The size query returns 0 for unsupported arguments.
 */
size_t swin_wattn_linear_bwd_weight_workspace_bytes(int tokens, int K, int N);
int swin_wattn_linear_bwd_weight(const void* dy, const void* x, void* dw, float* db, int tokens, int K, int N,
                                 int dtype, int accumulate, void* workspace, size_t workspace_bytes, int* status,
                                 struct CUstream_st* stream);

/*
 * A stack of weight updates made near orthogonal by Newton-Schulz products, for an optimiser
 * that steps along U V^T of its momentum G = U S V^T instead of along G. Per matrix:
 *   X = G / (|G|_F + eps), then `steps` times X <- a X + (b A + c A^2) X, A = X X^T,
 *   (a, b, c) = (3.4445, -4.7750, 2.0315);   out = scale * X
 * (on the side of the smaller dimension, which gives the same). Every singular value is
 * taken towards [0.7, 1.2]; U and V are kept.
 *   g      [count, rows, cols], fp32 or bf16 by `dtype` (SWIN_WATTN_FP32 or
 *          SWIN_WATTN_BF16), contiguous, 4- or 2-byte aligned;
 *   out    bf16 [count, rows, cols], 2-byte aligned, written (16-byte aligned with cols a
 *          multiple of 8 is the fast case); must not overlap g;
 *   count  in [0, 65535] (0: nothing is done); rows, cols in [1, 16384];
 *   steps  in [1, 20]; eps finite and > 0, not subnormal; scale finite, zero or
 *          at least 2^-100 in size;
 *   workspace  caller-owned device memory of at least
 *          swin_wattn_orthogonalize_workspace_bytes(count, rows, cols) bytes, 256-byte
 *          aligned, overwritten; one call at a time per workspace.
 * A and the polynomial are held in fp16 (scaled; the values are bounded), X in two fp16 parts of
 * 22 bits together, products are accumulated in fp32. Five steps end within 2e-3 (relative
 * 2-norm, before the rounding of the result to bf16) of the exact iteration where the smaller
 * side is at least 64, whatever G's rank and singular values: directions that G does not have
 * stay empty. Fewer rows average their roundings less: within 4e-3 from 32, 6e-3 from 2. Each
 * further step multiplies what the earlier ones left in directions still rising by up to 3.44, as
 * it does to G's own rounding: 4e-3 after seven steps, 1.1e-2 after ten (smaller side at least 64).
 * (The largest found over ranks from 1, singular values from flat to k^-2, and two groups of them up to
 * 1e4 apart.) Where |G| is far below eps, X is small from the start; its entries are held to
 * 2^-39. The norm is summed in fp32, in three ranges of size so that no square overflows or is
 * lost; subnormal values count as zero, and a norm beyond the largest fp32 gives zeros. A matrix
 * with a NaN or an infinity gives NaN and leaves the others of the stack alone; a zero matrix
 * gives zeros.
 * One launch where the smaller side is at most 128 and the larger at most 2048, else
 * 2 + 3 * steps, or 2 + 4 * steps where the longer side is split; nothing is allocated.
 * Deterministic. Errors: INVALID_ARG for the scalars, overlaps, a small workspace or a pointer
 * that the current device cannot address as its own; MISALIGNED; UNSUPPORTED for sizes out of
 * range. The size query returns 0 for unsupported arguments.
 */
size_t swin_wattn_orthogonalize_workspace_bytes(int count, int rows, int cols);
int swin_wattn_orthogonalize(const void* g, void* out, int count, int rows, int cols, int dtype, int steps, float eps,
                             float scale, void* workspace, size_t workspace_bytes, int* status,
                             struct CUstream_st* stream);

/*
 * The residual sum around a block, with its gate, its stochastic depth and the norms on both sides
 * (NVIDIA Swin talk, section 1: a block's LayerNorm and shortcut):
 *   u = post(f), or f without post;   y = alpha x + keep[sample] gate[channel] u;   h = pre(y)
 * pre is the norm before the next block (its output feeds that block's products), post the norm after
 * this one. norm(v) = vhat w + b, vhat by `kind` (SWIN_WATTN_NORM_*) over the C channels of a token.
 *   x      [tokens, C], the residual stream, bf16 or fp32 by `dtype`;
 *   f      bf16 [tokens, C], the block's output, or NULL: then h = pre(x), and y, post_*, gate
 *          and keep are NULL and alpha is not used;
 *   pre_w, pre_b, post_w, post_b  fp32 [C], 4-byte aligned; pre_w NULL: no pre norm (h is not
 *          written); post_w NULL: no post norm; pre_b, post_b NULL: no bias;
 *   gate   fp32 [C] or NULL (1);   keep  fp32 [samples] or NULL (1): a factor for each run of
 *          tokens / samples tokens (stochastic depth: 0, or 1 / the probability of keeping);
 *   y      [tokens, C] of x's dtype, written; may be x itself;
 *   h      bf16 [tokens, C], written; overlaps nothing;
 *   tokens in [0, 2^31 - 1024] (0: nothing is done); C a multiple of 8 in [8, 8192]; samples divides tokens;
 *   alpha, eps finite, eps a normal number above 0.
 * Device pointers of the current device, 16-byte aligned unless stated. Arithmetic in fp32: the mean is
 * taken out before squares are summed; h is normalised from y before y is rounded. Squares are summed in
 * fp32: rows are right while C times the largest square is below 3e38. NaN and infinities stay in
 * their token (0 * NaN is NaN: a dropped sample's f counts). One launch, nothing is allocated. Deterministic: the order of
 * a row's sums depends on the sizes, tokens among them, alone.
 * Errors: INVALID_ARG, MISALIGNED, UNSUPPORTED (C or tokens out of range).
 */
int swin_wattn_block_norm(const void* x, const void* f, const float* pre_w, const float* pre_b, const float* post_w,
                          const float* post_b, const float* gate, const float* keep, void* y, void* h, int tokens, int C,
                          int samples, int dtype, int kind, float alpha, float eps, struct CUstream_st* stream);

/*
 * Its gradients, for the gradients dh of h and dy of y (that of y's other uses):
 *   y      the forward's y (or x, without f); f, pre_w, post_w, post_b, gate, keep, alpha, kind, eps as there;
 *   dh     bf16 [tokens, C]; NULL exactly where pre_w is;
 *   dy     [tokens, C] of the stream's dtype, or NULL for none;
 *   dx     [tokens, C] of the stream's dtype, written; may be dy itself;
 *   df     bf16 [tokens, C], written; NULL exactly where f is;
 *   dpre_w, dpre_b, dpost_w, dpost_b, dgate  fp32 [C], written or added to (accumulate); NULL: not
 *          computed. Only those of what is there may be given;
 *   workspace  at least swin_wattn_block_norm_bwd_workspace_bytes(tokens, C) bytes, 256-byte aligned,
 *          overwritten; one call at a time per workspace.
 * With no tokens the parameter gradients are zeroed (left as they are when accumulating). The channel sums are
 * taken in fp32 in an order that depends on the sizes alone: deterministic. Two launches (one without
 * parameter gradients); nothing is allocated.
 */
size_t swin_wattn_block_norm_bwd_workspace_bytes(int tokens, int C);
int swin_wattn_block_norm_bwd(const void* y, const void* f, const void* dh, const void* dy, const float* pre_w,
                              const float* post_w, const float* post_b, const float* gate, const float* keep, void* dx,
                              void* df, float* dpre_w, float* dpre_b, float* dpost_w, float* dpost_b, float* dgate,
                              int tokens, int C, int samples, int dtype, int kind, float alpha, float eps, int accumulate,
                              void* workspace, size_t workspace_bytes, struct CUstream_st* stream);

/*
 * The norm over all gradients of a model and their clipping, between the gradients and the weight updates:
 *   n = scale * sqrt(sum of g^2 over all tensors),   out = g * scale * min(1, max_norm / (n + eps))
 * swin_wattn_clip_plan looks at the tensors once and writes a list of them, cut into pieces, into `list`, the caller's
 * device memory of at least swin_wattn_clip_list_bytes(sizes, dtypes, count) bytes, 256-byte aligned (32 bytes for some 2048
 * to 16384 elements); it copies to the device and waits for `stream`, so not during a capture. The tensors and the
 * list have to stay where they are while the plan or a graph made with it is used, the tensors' values may change.
 * The plan itself is host memory: swin_wattn_clip_destroy touches no device.
 *   grads, outs  `count` device pointers each, at any multiple of their element size; outs[i] may be
 *          grads[i] itself (in place), else it overlaps nothing; no tensor may be written twice;
 *   sizes  elements of each (0: the tensor is skipped); dtypes  SWIN_WATTN_FP32 or SWIN_WATTN_BF16 of each.
 * swin_wattn_clip_grad_norm runs it: norm (device fp32, or NULL) receives n; max_norm >= 0, scale > 0 and
 * eps >= 0, finite; workspace at least swin_wattn_clip_workspace_bytes() bytes, 256-byte aligned,
 * overwritten, one call at a time per workspace. The squares are summed in two fp32 parts (in fp32 within 64 bytes), those
 * that fp32 does not hold in 64 bits, in an order that depends on the sizes alone: deterministic, without overflow. Where n
 * or the factor leaves fp32's normal range both are formed in 64 bits: a finite n above it is stored as an infinity, and the
 * values are scaled all the same. Subnormal gradients and results are kept. A NaN anywhere makes n and every out NaN; an
 * infinity makes n infinite, the finite values 0 and itself NaN. Two launches;
 * where all are in place and their factor is 1 nothing is written. Errors: BAD_PLAN; INVALID_ARG, MISALIGNED as
 * above; INVALID_ARG also where the plan's device is not the current one.
 */
typedef struct swin_wattn_clip_s* swin_wattn_clip_t;
size_t swin_wattn_clip_list_bytes(const int64_t* sizes, const int* dtypes, int count);
int swin_wattn_clip_plan(swin_wattn_clip_t* plan, const void* const* grads, void* const* outs, const int64_t* sizes,
                         const int* dtypes, int count, void* list, size_t list_bytes, struct CUstream_st* stream);
size_t swin_wattn_clip_workspace_bytes(void);
int swin_wattn_clip_grad_norm(swin_wattn_clip_t plan, float max_norm, float scale, float eps, float* norm, void* workspace,
                              size_t workspace_bytes, struct CUstream_st* stream);
int swin_wattn_clip_destroy(swin_wattn_clip_t plan);

/*
 * Microscaled 4-bit operands: E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the
 * even one in the low half, rows of K / 2 bytes; and a scale for each block of a row, by `format`:
 *   NVFP4: s = E4M3(amax / 6 / ts), q = E2M1(x / (s ts)), blocks of 16, ts the tensor's scale;
 *   MXFP4: s = 2^(floor(log2 amax) - 2), at least 2^-127, q = E2M1(x / s), blocks of 32 (OCP MX);
 * amax the block's largest magnitude; to nearest, ties to even, saturated. A block with a NaN or an
 * infinity gets a NaN scale and reads back as NaN.
 * The scales lie in tiles of 128 rows by 4 blocks, as the tensor core reads them: row r and block j of tile
 * (R, J) at byte (R * ceil(blocks / 4) + J) * 512 + (r % 32) * 16 + (r / 32) * 4 + j; rows and blocks past the end
 * hold zeros. swin_wattn_fp4_scale_bytes gives their size (0: unsupported sizes).
 *   x      [rows, K], fp32 or bf16 by `dtype`; codes [rows, K / 2] bytes, written; scales, written;
 *   tensor_scale  NVFP4: device fp32. scale_given: read, between 2^-100 and 2^100; else written: the
 *          smallest power of two with max |x| <= 2688 ts (finite x; at least 2^-90), with which every rounding is
 *          that of the exact quotient and every value read back is exact in bf16. MXFP4: NULL;
 *   rows   in [0, 2^31 - 1024]; K a multiple of 32 in [32, 32768];
 *   workspace  needed for a scale that is not given: swin_wattn_fp4_workspace_bytes() bytes, 256-byte
 *          aligned, overwritten, one call at a time per workspace.
 * swin_wattn_fp4_dequantize reads them back, q (s ts) or q s: out [rows, K], fp32 or bf16 by `dtype`; fp32 is rounded as the
 * two products are, bf16 once more.
 * Device pointers of the current device, 16-byte aligned (tensor_scale 4). One launch, or two for a scale that is
 * not given; deterministic; nothing is allocated.
 */
size_t swin_wattn_fp4_scale_bytes(int rows, int K, int format);
size_t swin_wattn_fp4_workspace_bytes(void);
int swin_wattn_fp4_quantize(const void* x, void* codes, void* scales, float* tensor_scale, int rows, int K, int format,
                            int dtype, int scale_given, void* workspace, size_t workspace_bytes,
                            struct CUstream_st* stream);
int swin_wattn_fp4_dequantize(const void* codes, const void* scales, const float* tensor_scale, void* out, int rows, int K,
                              int format, int dtype, struct CUstream_st* stream);

/*
 * A dense layer on such operands (swin_wattn_linear's, for serving):
 *   y = residual + act(ts_x ts_w sum over k of (q_x s_x)(q_w s_w) + b)
 * x [tokens, K] and w [N, K] as codes, scales and tensor scales of one format (tensor scales NULL for MXFP4); b,
 * residual, y, act and status as for swin_wattn_linear; y must not overlap the operands.
 * K a multiple of 32, N a multiple of 8, up to 32768. The tensor cores multiply the 4-bit values with their block
 * scales and accumulate in fp32; the rest is fp32, y is rounded once. One launch; deterministic.
 */
int swin_wattn_linear_fp4(const void* x_codes, const void* x_scales, const float* x_tensor_scale, const void* w_codes,
                          const void* w_scales, const float* w_tensor_scale, const float* b, const void* residual, void* y,
                          int tokens, int K, int N, int format, int act, int* status, struct CUstream_st* stream);

/*
 * The same for an x [tokens, K] that is not quantised, fp32 or bf16 by `dtype`: it is quantised into the workspace, as
 * swin_wattn_fp4_quantize would (x_tensor_scale: the given scale of NVFP4, or NULL: taken from x; NULL for MXFP4).
 *   workspace  at least swin_wattn_linear_fp4_workspace_bytes(tokens, K, N, format, scale_given) bytes, 256-byte aligned,
 *          overwritten, one call at a time per workspace; NULL where that is 0 (scale_given: whether x_tensor_scale
 *          is; the query also returns 0 for unsupported arguments).
 * Two launches, or three for a scale that is taken from x; one, without a workspace, where 64 tokens at most, with no scale to
 * take, are quantised by the product itself (an estimate of both forms decides, which counts what a launch costs the
 * host; in a graph 49 tokens and more of a wide N are up to 2 us shorter as swin_wattn_fp4_quantize and
 * swin_wattn_linear_fp4).
 */
size_t swin_wattn_linear_fp4_workspace_bytes(int tokens, int K, int N, int format, int scale_given);
int swin_wattn_linear_fp4_of(const void* x, const float* x_tensor_scale, const void* w_codes, const void* w_scales,
                             const float* w_tensor_scale, const float* b, const void* residual, void* y, int tokens, int K,
                             int N, int format, int dtype, int act, void* workspace, size_t workspace_bytes, int* status,
                             struct CUstream_st* stream);

/*
 * Forward on 8-bit operands (7x7 windows, a SWIN_WATTN_BF16 plan): the attention of
 * q = scale_q * q8, k = scale_k * k8, v = scale_v * v8 for
 *   qkv8   device, 16-byte aligned: [B,H,W,3C] OCP FP8 E4M3 values, one byte each, in the
 *          token layout of qkv (q | k | v channels of a token);
 *   scale_q, scale_k, scale_v  one fp32 scale per tensor, finite and positive;
 *   out    device, 16-byte aligned: [B,H,W,C] bf16, written.
 * q8 k8^T runs on the 8-bit tensor cores (exact products, fp32 accumulation), the bias and
 * the shift mask are those of the plan, P is rounded to fp16, and v8 is widened exactly to
 * fp16 for P V: the result is the attention of the decoded values to the tolerance of
 * swin_wattn_fwd, with 3C instead of 6C bytes of qkv read per token (the pages take the
 * Swin GEMMs to 8 bits for inference, NVIDIA Swin talk section 3; here the attention's
 * operands). One kernel launch. UNSUPPORTED for another window size or dtype,
 * INVALID_ARG for a bad scale, and the pointer errors of swin_wattn_fwd.
 */
int swin_wattn_fwd_fp8(swin_wattn_plan_t plan, const void* qkv8, float scale_q, float scale_k, float scale_v,
                       void* out, struct CUstream_st* stream);

/*
 * Choose the plan's forward kernel (SWIN_WATTN_KERNEL_*): MMA_SYNC (every window size and
 * dtype) or TCGEN05 (the tensor-memory kernels: window 7 or 12, bf16). Both compute the
 * same function to the same tolerance. AUTO, the default, takes the faster as measured:
 * TCGEN05 for 12 x 12 windows when the plan has at least 16 window-heads per SM
 * (B * windows * heads >= 16 * SMs), else MMA_SYNC. Asking for TCGEN05 where it does not
 * apply returns SWIN_WATTN_ERR_UNSUPPORTED and leaves the plan unchanged. Host-side only;
 * call it between launches.
 */
int swin_wattn_set_fwd_kernel(swin_wattn_plan_t plan, int kernel);

/* The forward kernel the plan launches (MMA_SYNC or TCGEN05), or -1 for a bad handle. */
int swin_wattn_fwd_kernel(swin_wattn_plan_t plan);

/*
 * Choose the plan's backward kernel (SWIN_WATTN_KERNEL_*): MMA_SYNC (window 4 or 7, both
 * dtypes) or TCGEN05 (the tensor-memory kernel: window 7, bf16). Both compute the same
 * gradients to the same tolerance and are deterministic. AUTO, the default, takes the
 * faster as measured: TCGEN05 where it applies, except at shifted layers whose window grid
 * is at most two windows wide (there half or more of the windows wrap at the right edge
 * and are gathered four rows at a time), else MMA_SYNC. UNSUPPORTED where the choice does
 * not apply (the plan is then unchanged). Host-side only; call it between launches.
 */
int swin_wattn_set_bwd_kernel(swin_wattn_plan_t plan, int kernel);

/* The backward kernel the plan launches (MMA_SYNC or TCGEN05), or -1 for a bad handle. */
int swin_wattn_bwd_kernel(swin_wattn_plan_t plan);

/*
 * Synchronise `stream` and report the plan's device error word: SWIN_WATTN_ERR_TIMEOUT
 * if a kernel's bounded wait on the tensor core (1 s) ran out since the last call, in
 * which case that launch's output is not valid; the word is cleared. Otherwise OK.
 */
int swin_wattn_device_status(swin_wattn_plan_t plan, struct CUstream_st* stream);

/* Free the plan's device memory (synchronises the device first). NULL is a no-op. */
int swin_wattn_destroy(swin_wattn_plan_t plan);

/* Static text for a status code. */
const char* swin_wattn_status_string(int status);

/* CUDA error text behind the calling thread's last SWIN_WATTN_ERR_CUDA ("" if none). */
const char* swin_wattn_last_error(void);

/* Kernel launches issued by the calling thread since the last reset (for accounting). */
uint64_t swin_wattn_launch_count(int reset);

#ifdef __cplusplus
}
#endif

#endif /* SWIN_WATTN_H */
