// Batched matrix products on the fifth-generation tensor cores, with the epilogues of a
// block's MLP, of its gradients and of the weight update:
//   D[b] (M x N) = A[b] (M x K) B[b]^T (N x K),   A, B 16-bit, fp32 accumulation.
// Each operand may be stored K-major (rows of K contiguous elements) or MN-major (K rows
// of M or N contiguous elements): the copy engine brings either into 128-byte-swizzled
// shared memory as it lies, and the matrix descriptor tells the tensor core which it is,
// so no operand is ever transposed in memory.
//
// One persistent CTA per SM (CG = 1) or one pair of CTAs on two SMs (CG = 2) walks output
// tiles of CG * 128 rows by NT <= 256 columns:
// * copy warp: per chunk of 64 along K, the CTA's 128 rows of A and NT / CG rows of B into a
//   ring of stages;
// * MMA warp, one thread (of the pair's first CTA): four K16 MMAs a chunk into one of two
//   tensor-memory accumulators;
// * sixteen epilogue warps, four per tensor-memory lane quadrant, taking 32-column slices in
//   turn: the epilogue's arithmetic in fp32 on a thread's 32 columns of one row, one
//   rounding, a swizzled staging tile per warp, a TMA store; while the next tile
//   accumulates. A second operand of the epilogue (residual, pre-activation, ...) arrives
//   by TMA ahead of its slice in the staging tile that the result is written over. (With eight
//   warps the issue slots were 42 % busy on the GELU epilogues, with sixteen 62 %: 50176 x 192 x
//   768 with GELU and pre-activation 41 -> 33 us. Coalesced stores by the warps instead of TMA
//   stores: 42 us.)
// A pair (CG = 2) reads each row of B once for 256 rows of A instead of 128: per chunk a CTA
// brings 128 + NT / 2 rows instead of 128 + NT, which is what the tensor cores need to run
// at full rate at NT = 256 (shared memory is both filled and read by the chunk).
//
// What bounds it, measured on one GB300 (of the measured 6797 GB/s and 1865 TFLOP/s): wide products
// the tensor cores (12561 x 6144 x 1536 with residual: 127.5 us, 1.00, of calls one after the other
// 147 us, 0.86, at the power limit; 8192^3: 599 us, 0.98);
// narrow K the memory (50176 x 192 x 768, two results: 31.5 us, 0.81); short K with a slope
// epilogue the epilogue warps' issue (12544 x 512 -> 2048: 34.9 us, 0.50, of which the last of six
// rounds of tiles is a sixth full); the smallest launches latency, some 3.5 us from one launch to
// the next (0.9 until the last grid's writes are seen, 0.9 to the first chunk, 0.6 for its
// product, 0.7 for the epilogue, 0.4 to leave).
// Every wait is bounded (1 s); a wait that runs out sets the caller's status word (when one
// is given) and the CTA leaves after its copies have landed and its tensor memory is freed.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "tc.cuh"

namespace swin {
namespace prod {

constexpr int kBM = 128;   // rows of A per CTA
constexpr int kKC = 64;    // K per chunk: one 128-byte row
constexpr int kSC = 32;    // columns per epilogue slice
constexpr int kMaxNT = 256;
constexpr int kMaxStages = 8;
constexpr int kABytes = kBM * 128;
constexpr uint32_t kSW128 = 2;  // descriptor layout: 128-byte swizzle
constexpr int kTmemCols = 512;  // two accumulators of up to 256 columns
// An fp32 result keeps its accuracy over a long K by accumulating at most this many chunks
// (32 MMAs) in tensor memory, whose additions truncate; the epilogue warps add such segments
// up in registers, rounding to nearest. On 50176 tokens the error against 64 bits is 4.8e-7
// (relative 2-norm), where one accumulation per tile of 33 chunks left 2.1e-6; an 8192^3 product
// takes 777 us instead of the 709 us of a bf16 result without segments. The sums over K, which are
// fp32 beside a bf16 result too, are taken out of tensor memory in the same segments (12544 tokens of
// sizes spread over six decades: 0.6e-6, or 1.2e-6 of terms of one sign, where one accumulation lost
// 1.5e-5 and 4.0e-5).
constexpr int kSegChunks = 8;

// Barriers: full and empty per stage, full and free per accumulator, the last commit, aux
// loads (up to four per epilogue warp), full and free per segment of kEpiGrad16's sums.
constexpr int kMaxAuxTiles = 4;
constexpr int kDFull = 2 * kMaxStages, kDFree = kDFull + 2, kDrain = kDFree + 2, kAux = kDrain + 1;
constexpr int kSumFull = kAux + kMaxAuxTiles * 16, kSumFree = kSumFull + 2, kNBar = kSumFree + 2;

enum Epi {
  kEpiAct = 0,     // bf16: aux + act(acc + bias), optionally acc + bias into a second result
  kEpiSlope = 1,   // bf16: acc * act'(aux)
  kEpiGrad32 = 2,  // fp32: [old +] acc, optionally the column sums of A^T (sum over K of A);
                   // where K is split, a result per split (of each matrix)
  kEpiGrad16 = 3,  // bf16: [aux +] acc, optionally the same sums
  // of the weight update (orthogonalize.cu), on fp16 operands:
  kEpiGram = 4,    // fp16: alpha * acc, after diag was added to the diagonal of acc
  kEpiPoly = 5,    // fp16: alpha * acc + beta * aux, likewise; and the gains of its diagonal
  // alpha * gain * acc, in bf16, or in two fp16 parts: its rounding, and what that leaves. One operand
  // is X in such parts, and K is walked once for each
  kEpiUpdate = 6
};
// Symmetric results, of which only the tiles and slices on and below the diagonal may be computed;
// those below are then stored a second time, transposed. The tiling says whether (tiling_cost).
__host__ __device__ constexpr bool symmetric(int epi) { return epi == kEpiGram || epi == kEpiPoly; }

// Warps: the epilogue's, MMA, copy. The fp32 gradient has eight epilogue warps, which hold 128
// running sums a thread, more than an even share of the registers: two idle warps complete a
// third warpgroup, which gives registers up (2 x 216 + 64 of the 3 x 168 that 384 threads are
// launched with).
__host__ __device__ constexpr int epi_warps(int epi) { return epi == kEpiGrad32 ? 8 : 16; }
__host__ __device__ constexpr int n_threads(int epi) { return epi == kEpiGrad32 ? 384 : 576; }

// Division of 0 <= n < 2^31 by a fixed d >= 1: n / d = (umulhi(n, mul) + n) >> shift. (The
// plain divisions of an item's number cost every epilogue warp a hundred instructions a tile,
// as many as a slice's own work.)
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t divisor) : d(divisor), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

struct Params {
  int M, N, NT;
  FastDiv n_mt, n_nt, n_splits;
  bool half;                // of a symmetric result
  FastDiv n_lower, per_nt;  // with half: tiles of a matrix that are computed; NT
  int n_items;  // batch * splits * n_mt * n_nt (or batch * n_lower), n fastest
  int chunks, chunks_per_split;
  int stages, stage_bytes;
  int off_out, warp_bytes, tiles, off_small, off_bar;  // tiles: a warp's staging tiles before that of pre
  uint32_t idesc, idesc_ones;
  int act;
  bool has_aux, has_pre;
  bool to_bf16;           // kEpiUpdate: bf16 instead of fp16 parts
  int part_chunks;        // kEpiUpdate: chunks of K of one part of X; B where gain_rows, else A
  const float* bias;      // kEpiAct: [N] or null
  const float* old;       // kEpiGrad32: [M, N] added to the product, or null
  float* k_sums;          // kEpiGrad*: [splits, M], or null
  bool add_k_sums;        // the sums are added to what k_sums holds
  float alpha, beta, diag;
  // fp32 [batch, gain_ld], gain_ld a multiple of 32: each diagonal entry of kEpiPoly's result over
  // its rounding, which is kEpiUpdate's factor of a row (gain_rows) or column
  float* gain;
  int gain_ld;
  bool gain_rows;
  __nv_bfloat16* raw_out;  // kEpiUpdate: plain stores (a row length the copy engine cannot address), or null
  int* status;
  uint64_t wait_ns;
  int fault;
};

// ---- pairs of CTAs ------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The two halves of the barrier, without memory ordering: for the end of a kernel, where a warp
// arrives once it has no more to do with the other CTA and the CTA waits before it leaves.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
}
// The address, in the cluster's shared memory, of this CTA's address `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t mbar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(mbar) : "memory");
}

template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t mbar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(mbar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(mbar)
        : "memory");
}
__device__ __forceinline__ void store_3d(const CUtensorMap* map, int c0, int c1, int c2, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(map),
               "r"(c0), "r"(c1), "r"(c2), "r"(src)
               : "memory");
}

// D[tmem] (+)= A B^T; a and b are the low words of the operands' descriptors, *_hi the high
// ones. (One thread issues every MMA: building whole descriptors there, some twenty
// instructions each, took 700 clocks a chunk where the tensor core takes 512 at N = 256.)
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                    bool accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.u32 p, %6, 0;\n mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.u32 p, %6, 0;\n mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// True in one lane of a converged warp. The MMA loop runs in the whole warp, with only the
// issue in this lane: the compiler then knows the operands uniform and keeps them in uniform
// registers (a chunk of four MMAs issues in 180 clocks; in a one-thread loop, in 260).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r));
  return r != 0;
}
// The words of a descriptor (tc::sdesc): low, address and lbo; high, sbo, version and layout.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | (lbo >> 4) << 16; }
__device__ __forceinline__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t layout) { return (sbo >> 4) | 1u << 14 | layout << 29; }
// Arrive on the mbarrier (of both CTAs of a pair) when every MMA issued so far has completed.
template <int CG>
__device__ __forceinline__ void commit(uint32_t mbar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
            mbar),
        "h"((uint16_t)3)
        : "memory");
  else
    tc::commit(mbar);
}
// The same, of the issuing CTA alone.
template <int CG>
__device__ __forceinline__ void commit_here(uint32_t mbar) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(mbar)
                 : "memory");
  else
    tc::commit(mbar);
}
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t dst) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst), "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  } else {
    tc::tmem_alloc<kTmemCols>(dst);
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t base) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(base), "n"(kTmemCols) : "memory");
  else
    tc::tmem_dealloc<kTmemCols>(base);
}

// Wait for a phase, as tc::mbar_wait; its clock is read only where the first try, which
// suspends the thread itself, has run out.
__device__ __forceinline__ bool wait(uint32_t mbar, uint32_t parity, uint64_t limit_ns) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred q;\n mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(ok)
      : "r"(mbar), "r"(parity)
      : "memory");
  return ok ? true : tc::mbar_wait(mbar, parity, limit_ns);
}
__device__ __forceinline__ bool warp_wait(uint32_t mbar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, wait(mbar, parity, limit_ns)) != 0;
}

// ---- activations --------------------------------------------------------------------
//
// Every smooth activation here is z * s(z) with s(-z) = 1 - s(z), so with t = |z| and
// h(t) = s(-t):   act(z) = max(z, 0) - t h(t),   s(z) = z > 0 ? 1 - h : h.
// This form keeps the relative accuracy of the small tail h and needs no sign handling.
// * GELU: h(t) = Phi(-t), the normal distribution function. log2 Phi(-t) is close to a
//   parabola, so h = 2^Q(t) with Q of degree 6, fitted (minimax, iteratively reweighted
//   least squares) on [0, 6]: |h / Phi(-t) - 1| < 5e-5 there, |t h - t Phi(-t)| < 7e-6
//   everywhere, a fortieth of a bf16 rounding; six multiply-adds and one exponential where
//   erff takes some twenty instructions. Q falls monotonically up to t = 15, where
//   t is cut, which also keeps infinities out of the polynomial; 2^Q is below the smallest normal
//   fp32, and so 0, from t = 13.9 on.
// * tanh-GELU: 0.5 (1 + tanh u) = 1 / (1 + exp(-2u)), so h = 1 / (1 + exp(2 u(t))).
// * SiLU: h = 1 / (1 + exp(t)).
// t is cut at 100 there: exp overflows to infinity and h is 0 long before.
// The minimum that cuts t propagates NaN, so a NaN input gives NaN.

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// z > 0 ? 1 : 0, subnormal z included (an ordinary comparison here is built to flush them).
__device__ __forceinline__ float step01(float z) {
  float r;
  asm("set.gt.f32.f32 %0, %1, 0f00000000;\n" : "=f"(r) : "f"(z));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

constexpr float kGeluCut = 15.0f, kSigmoidCut = 100.0f;
constexpr float kTanhA = 0.7978845608028654f, kTanhB = 0.044715f;  // u(z) = A (z + B z^3)

// t = min(|z|, cut), NaN kept, and h(t), for two values.
template <int ACT>
__device__ __forceinline__ void act_tail(float2 z, float2& t, float2& h) {
  if constexpr (ACT == SWIN_WATTN_ACT_GELU) {
    t = make_float2(min_nan(fabsf(z.x), kGeluCut), min_nan(fabsf(z.y), kGeluCut));
    float2 q = splat(2.29900633712532e-05f);
    q = __ffma2_rn(q, t, splat(-0.0006111000548116863f));
    q = __ffma2_rn(q, t, splat(0.007195565849542618f));
    q = __ffma2_rn(q, t, splat(-0.05118533596396446f));
    q = __ffma2_rn(q, t, splat(-0.46127191185951233f));
    q = __ffma2_rn(q, t, splat(-1.1501742601394653f));
    q = __ffma2_rn(q, t, splat(-1.000064730644226f));
    h = make_float2(fast_exp2(q.x), fast_exp2(q.y));
  } else {
    t = make_float2(min_nan(fabsf(z.x), kSigmoidCut), min_nan(fabsf(z.y), kSigmoidCut));
    float2 e;  // the exponent, in powers of two
    if constexpr (ACT == SWIN_WATTN_ACT_GELU_TANH) {
      constexpr float kA2 = 2.0f * kTanhA * kLog2e;
      e = __fmul2_rn(t, __ffma2_rn(__fmul2_rn(t, t), splat(kA2 * kTanhB), splat(kA2)));
    } else {
      e = __fmul2_rn(t, splat(kLog2e));
    }
    h = make_float2(fast_rcp(1.0f + fast_exp2(e.x)), fast_rcp(1.0f + fast_exp2(e.y)));
  }
}

template <int ACT>
__device__ __forceinline__ float2 act_value(float2 z) {
  if constexpr (ACT == SWIN_WATTN_ACT_NONE) return z;
  if constexpr (ACT == SWIN_WATTN_ACT_RELU) return make_float2(max_nan(z.x, 0.0f), max_nan(z.y, 0.0f));
  float2 t, h;
  act_tail<ACT>(z, t, h);
  return __ffma2_rn(make_float2(-t.x, -t.y), h, make_float2(fmaxf(z.x, 0.0f), fmaxf(z.y, 0.0f)));
}

// act'(z) = s + z s'(z). With n = h - t s'(t) it is 1 - n for z > 0 and n for z < 0, that is
// 1/2 + copysign(1/2 - n, z). GELU: s' = phi, the normal density; the others:
// s' = s (1 - s) (2 u)', and s (1 - s) = h (1 - h).
template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 z) {
  if constexpr (ACT == SWIN_WATTN_ACT_RELU) return make_float2(step01(z.x), step01(z.y));
  float2 t, h, s;
  act_tail<ACT>(z, t, h);
  if constexpr (ACT == SWIN_WATTN_ACT_GELU) {
    // phi(t) = 2^(-t^2 log2(e) / 2 - log2 sqrt(2 pi))
    const float2 e = __ffma2_rn(__fmul2_rn(t, t), splat(-0.5f * kLog2e), splat(-1.3257480647361595f));
    s = make_float2(fast_exp2(e.x), fast_exp2(e.y));
  } else {
    s = __fmul2_rn(h, fsub2(splat(1.0f), h));
    if constexpr (ACT == SWIN_WATTN_ACT_GELU_TANH)
      s = __fmul2_rn(s, __ffma2_rn(__fmul2_rn(t, t), splat(6.0f * kTanhA * kTanhB), splat(2.0f * kTanhA)));
  }
  const float2 d = __ffma2_rn(t, s, __ffma2_rn(h, splat(-1.0f), splat(0.5f)));  // 1/2 - n
  return __fadd2_rn(splat(0.5f), make_float2(copysignf(d.x, z.x), copysignf(d.y, z.y)));
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// a[lane]
__device__ __forceinline__ float of_lane(const uint32_t (&a)[32], int lane) {
  uint32_t t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = lane & 16 ? a[i + 16] : a[i];
#pragma unroll
  for (int n = 8; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = lane & n ? t[i + n] : t[i];
  return __uint_as_float(t[0]);
}

// Tiles of `rows` x NT on or below the diagonal in row mt of tiles.
__host__ __device__ __forceinline__ int lower_tiles(int mt, int rows, int NT, int n_nt, const FastDiv& per_nt) {
#ifdef __CUDA_ARCH__
  const int n = per_nt.quotient((mt + 1) * rows + NT - 1);
#else
  const int n = ((mt + 1) * rows + NT - 1) / NT;
#endif
  return n < n_nt ? n : n_nt;
}

// Bytes of one staging tile (32 rows x 32 columns) of an epilogue.
__host__ __device__ constexpr int tile_bytes(int epi) { return epi == kEpiGrad32 ? 4096 : 2048; }
// Staging tiles of an epilogue warp: with a second operand (aux) up to four, for the store of
// the last slice, this slice, and two loads ahead, or two where K is long; else two, or one
// where K is long; and one more for a second result (pre). Where K is long a tile's product
// takes longer than its epilogue, and shared memory is worth more in the ring: at 8192^3 a
// pair runs at 1580 TFLOP/s with four stages, 1750 with five.

template <int CG, bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(n_threads(EPI), 1)
    product_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                   const __grid_constant__ CUtensorMap out_map, const __grid_constant__ CUtensorMap aux_map,
                   const __grid_constant__ CUtensorMap pre_map, const Params p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  pdl_launch_dependents();
  const uint32_t smem0 = smem_u32(smem);
  if ((smem0 & 1023u) != 0) {  // the swizzled tiles need the declared alignment
    if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, 1);
    return;
  }
  const uint32_t bar0 = smem0 + p.off_bar;
  auto full_bar = [&](int st) { return bar0 + 8 * st; };
  auto empty_bar = [&](int st) { return bar0 + 8 * (kMaxStages + st); };
  auto dfull_bar = [&](int b) { return bar0 + 8 * (kDFull + b); };
  auto dfree_bar = [&](int b) { return bar0 + 8 * (kDFree + b); };
  auto sum_full_bar = [&](int s) { return bar0 + 8 * (kSumFull + (s & 1)); };
  auto sum_free_bar = [&](int s) { return bar0 + 8 * (kSumFree + (s & 1)); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + p.off_bar + 8 * kNBar);
  const int stages = p.stages;
  constexpr int kEW = epi_warps(EPI), kMMA = kEW, kCOPY = kEW + 1;
  constexpr int kPerQuad = kEW / 4, kSlices = kMaxNT / kSC / kPerQuad;  // warps per quadrant, slices per warp
  constexpr bool kSums = EPI == kEpiGrad32 || EPI == kEpiGrad16;
  constexpr int kSeg = EPI == kEpiGrad32 ? kSegChunks : 1 << 30;
  // The sums of a first-column tile take columns of their own: one set a segment of an fp32 result,
  // two in turn beside a bf16 one, whose sums alone are in segments. They lie behind the tile's
  // columns where there is room, else in the other accumulator's first columns.
  constexpr int kSumCols = 16 * CG;
  const bool sums_aside = p.NT + (EPI == kEpiGrad16 ? 2 : 1) * kSumCols > kMaxNT;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = CG == 2 ? (int)cluster_rank() : 0;
  const int group = blockIdx.x / CG, n_groups = gridDim.x / CG;

  // Work item -> first row and column of this CTA's part, first and last chunk, batch or split.
  struct Item {
    int m0, n0, c0, c1, nt, b, split;
  };
  auto decode = [&](int it) {
    Item w;
    if (symmetric(EPI) && p.half) {
      w.b = p.n_lower.quotient(it);
      w.nt = it - w.b * p.n_lower.d;
      int mt = 0;
      for (int n; w.nt >= (n = lower_tiles(mt, CG * kBM, p.NT, p.n_nt.d, p.per_nt)); ++mt) w.nt -= n;
      w.m0 = (mt * CG + rank) * kBM;
      w.n0 = w.nt * p.NT;
      w.split = w.c0 = 0;
      w.c1 = p.chunks;
      return w;
    }
    const uint32_t r1 = p.n_nt.quotient(it), r2 = p.n_mt.quotient(r1);
    w.nt = it - r1 * p.n_nt.d;
    const int mt = r1 - r2 * p.n_mt.d;
    w.b = p.n_splits.quotient(r2);
    w.split = r2 - w.b * p.n_splits.d;
    w.m0 = (mt * CG + rank) * kBM;
    w.n0 = w.nt * p.NT;
    w.c0 = w.split * p.chunks_per_split;
    w.c1 = min(w.c0 + p.chunks_per_split, p.chunks);
    return w;
  };

  if (warp == kMMA) tmem_alloc<CG>(smem_u32(tmem_slot));
  if (tid == 0) {
    for (int st = 0; st < stages; ++st) {
      tc::mbar_init(full_bar(st), 1);
      tc::mbar_init(empty_bar(st), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(dfull_bar(b), 1);
      tc::mbar_init(dfree_bar(b), kEW * CG);
    }
    for (int b = 0; b < kMaxAuxTiles * kEW; ++b) tc::mbar_init(bar0 + 8 * (kAux + b), 1);
    tc::mbar_init(bar0 + 8 * kDrain, 1);
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(sum_full_bar(b), 1);
      tc::mbar_init(sum_free_bar(b), 4 * CG);  // the warps of an epilogue's first part
    }
    tc::mbar_init_fence();
  }
  if constexpr (kSums) {
    // 16 rows x 16 of K, all ones (any layout): the B operand that sums A over K
    if (tid < 128) reinterpret_cast<uint32_t*>(smem + p.off_small)[tid] = 0x3F803F80u;
    tc::fence_proxy_async();
  }
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // The prologue above touches only this CTA's shared and tensor memory, so it may overlap
  // the previous kernel on the stream; every global access comes after this wait.
  pdl_wait();
  int bad = 0;
  if (warp >= kEW) {
    if constexpr (EPI == kEpiGrad32) tc::setmaxnreg_dec<64>();
    if (warp == kCOPY) {
      if (lane == 0) {
        int st = 0;
        uint32_t ph = 0, first = 1;
        // a pair's loads all complete on the first CTA's barriers
        const uint32_t full0 = CG == 2 ? map_to_rank(full_bar(0), 0) : full_bar(0);
        for (int it = group; it < p.n_items && !bad; it += n_groups) {
          const Item w = decode(it);
          const int nb0 = w.n0 + rank * (p.NT / CG);
          for (int c = w.c0; c < w.c1; ++c) {
            int kc = c * kKC, ba = w.b, bb = w.b;
            if constexpr (EPI == kEpiUpdate) {
              // the smaller part first: added to the larger one's sum it would lose its low bits
              const bool low = c < p.part_chunks;
              if (!low) kc -= p.part_chunks * kKC;
              (p.gain_rows ? bb : ba) = 2 * w.b + (low ? 1 : 0);
            }
            if (!first && !wait(empty_bar(st), ph ^ 1, p.wait_ns)) {
              bad = 1;
              break;
            }
            const uint32_t base = smem0 + st * p.stage_bytes;
            const uint32_t fb = full0 + 8 * st;
            if (rank == 0) tc::mbar_expect_tx(full_bar(st), CG * p.stage_bytes);
            if constexpr (AMN) {
#pragma unroll
              for (int j = 0; j < kBM / 64; ++j)
                load_3d<CG>(base + j * 8192, &a_map, w.m0 + 64 * j, kc, ba, fb);
            } else {
              load_3d<CG>(base, &a_map, kc, w.m0, ba, fb);
            }
            if constexpr (BMN) {
              // whole boxes of 64 columns: the last one may bring some that belong to the next part
              for (int j = 0; j * 64 < p.NT / CG; ++j)
                load_3d<CG>(base + kABytes + j * 8192, &b_map, nb0 + 64 * j, kc, bb, fb);
            } else {
              load_3d<CG>(base + kABytes, &b_map, kc, nb0, bb, fb);
            }
            if (++st == stages) {
              st = 0;
              ph ^= 1;
              first = 0;
            }
          }
        }
        // every load issued has landed before the CTA leaves (the second CTA of a pair is held
        // by the cluster barrier below until the first has seen its bytes too)
        if (rank == 0)
          for (int s2 = 0; s2 < (first ? st : stages); ++s2)
            tc::mbar_wait(full_bar(s2), s2 < st ? ph : ph ^ 1, p.wait_ns);
      }
      __syncwarp();
    } else if (warp == kMMA) {
      if (rank == 0) {
        constexpr uint32_t kHi = desc_hi(1024, kSW128), kOnesHi = desc_hi(256, 0);
        // along K by 16: K-major, 32 bytes further in the 128-byte row; MN-major, 16 rows
        // further, blocks of 64 of M or N 8192 bytes apart
        constexpr uint32_t kAStep = (AMN ? 2048 : 32) >> 4, kBStep = (BMN ? 2048 : 32) >> 4;
        const uint32_t a0 = desc_lo(smem0, AMN ? 8192 : 16), b0 = desc_lo(smem0 + kABytes, BMN ? 8192 : 16);
        const uint32_t ones_lo = desc_lo(smem0 + p.off_small, 128);
        const uint32_t stage_step = p.stage_bytes >> 4, idesc = p.idesc;
        [[maybe_unused]] const uint32_t idesc_ones = p.idesc_ones;
        int st = 0, g = 0;  // ring stage; accumulations begun
        [[maybe_unused]] int q = 0;  // segments of kEpiGrad16's sums begun
        uint32_t ph = 0;
        bool prev_ones = false;
        for (int it = group; it < p.n_items && !bad; it += n_groups) {
          const Item w = decode(it);
          const bool ones = kSums && p.k_sums != nullptr && w.nt == 0;
          const bool ones_aside = ones && sums_aside;
          for (int s0 = w.c0; s0 < w.c1 && !bad; s0 += kSeg, ++g) {
            const int s1 = min(s0 + kSeg, w.c1), buf = g & 1;
            const uint32_t acc = tmem + buf * kMaxNT;
            const uint32_t sums0 = ones_aside ? tmem + (buf ^ 1) * kMaxNT : acc + p.NT;
            [[maybe_unused]] uint32_t sums = sums0;
            if (g >= 2 && !warp_wait(dfree_bar(buf), ((g >> 1) - 1) & 1, p.wait_ns)) {
              bad = 1;
              break;
            }
            // where the other accumulator holds sums, its own epilogue has to be over before,
            // and this one's before the next begins
            if (g >= 1 && (ones_aside || prev_ones) && !warp_wait(dfree_bar(buf ^ 1), ((g - 1) >> 1) & 1, p.wait_ns)) {
              bad = 1;
              break;
            }
            prev_ones = ones_aside;
            for (int c = s0; c < s1; ++c) {
              if (!warp_wait(full_bar(st), ph, p.wait_ns)) {
                bad = 1;
                break;
              }
              const int of_sums = EPI == kEpiGrad16 ? (c - s0) % kSegChunks : c - s0;  // chunk of its segment
              if (EPI == kEpiGrad16 && ones && of_sums == 0) {
                if (q >= 2 && !warp_wait(sum_free_bar(q), ((q >> 1) - 1) & 1, p.wait_ns)) {
                  bad = 1;
                  break;
                }
                sums = sums0 + (q & 1) * kSumCols;
                ++q;
              }
              tc::fence_after_sync();
              const uint32_t a = a0 + st * stage_step, b = b0 + st * stage_step;
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  mma<CG>(acc, a + kk * kAStep, kHi, b + kk * kBStep, kHi, idesc, c > s0 || kk > 0);
                  if (kSums && ones)
                    mma<CG>(sums, a + kk * kAStep, kHi, ones_lo, kOnesHi, idesc_ones, of_sums > 0 || kk > 0);
                }
                commit<CG>(empty_bar(st));
                if (EPI == kEpiGrad16 && ones && (of_sums == kSegChunks - 1 || c == s1 - 1)) commit<CG>(sum_full_bar(q - 1));
#ifdef SWIN_WATTN_FAULT_INJECTION
                if (!(p.fault == kFaultGemm && g == 0))
#endif
                  if (c == s1 - 1) commit<CG>(dfull_bar(buf));
              }
              __syncwarp();
              if (++st == stages) {
                st = 0;
                ph ^= 1;
              }
            }
          }
        }
        // every MMA issued has completed before the tensor memory is released
        if (elect_one()) commit_here<CG>(bar0 + 8 * kDrain);
        __syncwarp();
        if (!warp_wait(bar0 + 8 * kDrain, 0, p.wait_ns)) bad = 1;
      }
      __syncwarp();
    }
  } else {
    if constexpr (EPI == kEpiGrad32) tc::setmaxnreg_inc<216>();
    // ==== epilogue warps ================================================================
    constexpr int kTile = tile_bytes(EPI);
    const int quad = warp & 3, part = warp >> 2;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
    unsigned char* wstage = smem + p.off_out + warp * p.warp_bytes;
    constexpr bool kHasAux = EPI != kEpiGrad32 && EPI != kEpiGram && EPI != kEpiUpdate;
    const bool aux = kHasAux && p.has_aux, pre = EPI == kEpiAct && p.has_pre;
    const bool parts = EPI == kEpiUpdate && !p.to_bf16;
    const int NB = p.tiles;
    const uint32_t aux0 = bar0 + 8 * (kAux + kMaxAuxTiles * warp);
    // the next slice whose second operand is to be requested: its item, decoded, and its columns,
    // and its staging tile
    int nx_it = group, nx_c0 = part * kSC, nx_end = 0, nx_row = 0, nx_n0 = 0, nx_b = 0, nx_tile = 0, issued = 0;
    auto next_item = [&]() {
      nx_end = 0;
      if (nx_it < p.n_items) {
        const Item w = decode(nx_it);
        nx_row = w.m0 + quad * 32;
        nx_n0 = w.n0;
        nx_b = w.b;
        nx_end = nx_row < p.M ? min(p.NT, p.N - w.n0) : 0;
        if (symmetric(EPI) && p.half) nx_end = min(nx_end, nx_row + kSC - w.n0);  // none above the diagonal
      }
    };
    auto request_next = [&]() {
      while (nx_it < p.n_items) {
        if (nx_c0 < nx_end) {
          if (lane == 0) {
            const uint32_t rb = aux0 + 8 * nx_tile;
            tc::mbar_expect_tx(rb, kTile);
            load_3d<1>(smem_u32(wstage + nx_tile * kTile), &aux_map, nx_n0 + nx_c0, nx_row, nx_b, rb);
          }
          ++issued;
          if (++nx_tile == NB) nx_tile = 0;
          nx_c0 += kPerQuad * kSC;
          return;
        }
        nx_it += n_groups;
        nx_c0 = part * kSC;
        next_item();
      }
    };
    if (aux) next_item();
    if (aux)
      for (int i = 0; i < max(NB - 2, 1); ++i) request_next();
    int g = 0, m = 0;                   // accumulations, slices of this warp
    [[maybe_unused]] int q = 0;         // segments of kEpiGrad16's sums
    int tile = 0;                       // the slice's staging tile
    uint32_t aux_phase = 0;             // of that tile's barrier
    for (int it = group; it < p.n_items && !bad; it += n_groups) {
      const Item w = decode(it);
      const int row0 = w.m0 + quad * 32, row = row0 + lane;
      // kEpiAct: the bias of the tile's columns in shared memory, for broadcast reads. Every
      // warp of a part writes the same values; two buffers, and the write waits for this
      // tile's accumulator, which is given out when every warp has left the tile before last.
      float* sbias = reinterpret_cast<float*>(smem + p.off_small) + (g & 1) * kMaxNT + part * kSC;
      float bt[kSlices];
      if constexpr (EPI == kEpiAct) {
#pragma unroll
        for (int i = 0; i < kSlices; ++i) {
          const int c = w.n0 + (part + kPerQuad * i) * kSC + lane;
          bt[i] = p.bias != nullptr && c < p.N ? p.bias[c] : 0.0f;
        }
      }
      float seg_sum[EPI == kEpiGrad32 ? kSlices : 1][32];  // kEpiGrad32: the segments' sum, a slice each
      if constexpr (EPI == kEpiGrad32) {
#pragma unroll
        for (int i = 0; i < kSlices; ++i)
#pragma unroll
          for (int e = 0; e < 32; ++e) seg_sum[i][e] = 0.0f;
      }
      float ones_sum = 0.0f;
      const bool adds_ones = kSums && p.k_sums != nullptr && w.nt == 0 && part == 0, ones = adds_ones && row0 < p.M;
      int buf = g & 1;
      const uint32_t sums = trow + (sums_aside ? (buf ^ 1) * kMaxNT : buf * kMaxNT + p.NT);  // of a single segment's tile
      if constexpr (EPI == kEpiGrad16) {
        // ahead of the product, which does not wait for more than two of them
        if (adds_ones) {
          for (int c = w.c0; c < w.c1; c += kSegChunks, ++q) {
            if (!warp_wait(sum_full_bar(q), (q >> 1) & 1, p.wait_ns)) {
              bad = 1;
              break;
            }
            tc::fence_after_sync();
            uint32_t s;
            tc::ld1_nowait(sums + (q & 1) * kSumCols, s);
            tc::wait_ld_then();
            tc::dep1(s);
            ones_sum += __uint_as_float(s);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
              if constexpr (CG == 2)
                arrive_cluster(map_to_rank(sum_free_bar(q), 0));
              else
                tc::mbar_arrive(sum_free_bar(q));
            }
          }
          if (bad) break;
        }
      }
      auto release = [&]() {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            arrive_cluster(map_to_rank(dfree_bar(buf), 0));
          else
            tc::mbar_arrive(dfree_bar(buf));
        }
        ++g;
      };
      for (int s0 = w.c0; s0 < w.c1; s0 += kSeg) {
        buf = g & 1;
        if (!warp_wait(dfull_bar(buf), (g >> 1) & 1, p.wait_ns)) {
          bad = 1;
          break;
        }
        tc::fence_after_sync();
        if constexpr (EPI == kEpiAct) {
#pragma unroll
          for (int i = 0; i < kSlices; ++i) sbias[kPerQuad * kSC * i + lane] = bt[i];
          __syncwarp();
        }
        if (EPI == kEpiGrad32 && ones) {
          uint32_t s;
          tc::ld1_nowait(trow + (sums_aside ? (buf ^ 1) * kMaxNT : buf * kMaxNT + p.NT), s);
          tc::wait_ld_then();
          tc::dep1(s);
          ones_sum += __uint_as_float(s);
        }
        if constexpr (EPI == kEpiGrad32) {
#pragma unroll
          for (int i = 0; i < kSlices; ++i) {
            const int c0 = (part + kPerQuad * i) * kSC;
            if (row0 < p.M && c0 < p.NT && w.n0 + c0 < p.N) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                uint32_t a[16];
                tc::ld16_wait(trow + buf * kMaxNT + c0 + h, a);
#pragma unroll
                for (int e = 0; e < 16; ++e) seg_sum[i][h + e] += __uint_as_float(a[e]);
              }
            }
          }
          release();
        } else if (s0 + kSeg >= w.c1) {
          break;
        }
      }
      if (bad) break;
      if (ones && row < p.M) {
        float* d = p.k_sums + (int64_t)w.split * p.M + row;
        *d = p.add_k_sums ? *d + ones_sum : ones_sum;
      }
#pragma unroll(EPI == kEpiGrad32 ? kSlices : 1)
      for (int si = 0; si < kSlices; ++si) {
        const int c0 = (part + kPerQuad * si) * kSC;
        if (!(row0 < p.M && c0 < p.NT && w.n0 + c0 < p.N)) continue;
        if (symmetric(EPI) && p.half && w.n0 + c0 > row0) continue;
        const bool mirror = symmetric(EPI) && p.half && w.n0 + c0 < row0;
        unsigned char* so = wstage + tile * kTile;
        unsigned char* sz = wstage + NB * kTile;
        if (aux) {
          // all stores but the last slice's (of two tiles, all) have read their tiles: load
          // ahead into the oldest
          if (lane == 0) {
            if (NB == 2)
              tc::bulk_wait_read<0>();
            else
              tc::bulk_wait_read<1>();
          }
          __syncwarp();
          request_next();
        }
        // kEpiUpdate: the factors of the slice's columns
        [[maybe_unused]] float4 factor[EPI == kEpiUpdate ? 8 : 1];
        if constexpr (EPI == kEpiUpdate) {
          const float* gain = p.gain + (int64_t)w.b * p.gain_ld;
          if (p.gain_rows) {
            const float f = row < p.M ? p.alpha * __ldcg(gain + row) : 0.0f;
#pragma unroll
            for (int c = 0; c < 8; ++c) factor[c] = make_float4(f, f, f, f);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 g = __ldcg(reinterpret_cast<const float4*>(gain + w.n0 + c0) + c);
              factor[c] = make_float4(p.alpha * g.x, p.alpha * g.y, p.alpha * g.z, p.alpha * g.w);
            }
          }
        }
        uint32_t a[32];
        if constexpr (EPI != kEpiGrad32) tc::ld32_wait(trow + buf * kMaxNT + c0, a);
        if (aux && !warp_wait(aux0 + 8 * tile, aux_phase, p.wait_ns)) {
          bad = 1;
          break;
        }
        // Before a tile without a second operand is written: the store that held it has read it.
        auto tile_free = [&]() {
          if (aux) return;
          if (lane == 0) {
            if (NB == 1)
              tc::bulk_wait_read<0>();
            else
              tc::bulk_wait_read<1>();
          }
          __syncwarp();
        };
        if constexpr (EPI == kEpiGrad32) {
          tile_free();
          const float* old = p.old != nullptr && row < p.M ? p.old + (int64_t)row * p.N + w.n0 + c0 : nullptr;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float4 v = make_float4(seg_sum[si][4 * c], seg_sum[si][4 * c + 1], seg_sum[si][4 * c + 2],
                                   seg_sum[si][4 * c + 3]);
            if (old != nullptr && w.n0 + c0 + 4 * c < p.N) {
              const float4 o = *reinterpret_cast<const float4*>(old + 4 * c);
              v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
            }
            *reinterpret_cast<float4*>(so + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
          }
        } else {
          unsigned char* sr = so + lane * 64;
          const int sw = (lane >> 1) & 3;
          auto at = [&](unsigned char* base, int c) { return reinterpret_cast<uint4*>(base + ((c ^ sw) << 4)); };
          auto pair = [&](int e) { return make_float2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])); };
          uint32_t o[16];  // the result, packed
          [[maybe_unused]] uint32_t low[EPI == kEpiUpdate ? 16 : 1];
          auto activate = [&](auto act) {
            constexpr int ACT = decltype(act)::value;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint4 r = make_uint4(0, 0, 0, 0);
              if (aux) r = *at(sr, c);
              const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
              if constexpr (EPI == kEpiAct) {
                const float4 b0 = reinterpret_cast<const float4*>(sbias + kPerQuad * kSC * si)[2 * c];
                const float4 b1 = reinterpret_cast<const float4*>(sbias + kPerQuad * kSC * si)[2 * c + 1];
                const float2 bb[4] = {make_float2(b0.x, b0.y), make_float2(b0.z, b0.w), make_float2(b1.x, b1.y),
                                      make_float2(b1.z, b1.w)};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float2 z = __fadd2_rn(pair(8 * c + 2 * q), bb[q]);
                  a[8 * c + 2 * q] = __float_as_uint(z.x);  // kept for the second result
                  a[8 * c + 2 * q + 1] = __float_as_uint(z.y);
                  float2 y = act_value<ACT>(z);
                  if (aux) y = __fadd2_rn(y, unpack_bf16(rr[q]));
                  o[4 * c + q] = pack_bf16(y.x, y.y);
                }
              } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  float2 y = pair(8 * c + 2 * q);
                  if constexpr (ACT != SWIN_WATTN_ACT_NONE) y = __fmul2_rn(y, act_slope<ACT>(unpack_bf16(rr[q])));
                  o[4 * c + q] = pack_bf16(y.x, y.y);
                }
              }
            }
          };
          if constexpr (EPI == kEpiAct || EPI == kEpiSlope) {
            switch (p.act) {
              case SWIN_WATTN_ACT_RELU: activate(std::integral_constant<int, SWIN_WATTN_ACT_RELU>()); break;
              case SWIN_WATTN_ACT_GELU: activate(std::integral_constant<int, SWIN_WATTN_ACT_GELU>()); break;
              case SWIN_WATTN_ACT_GELU_TANH: activate(std::integral_constant<int, SWIN_WATTN_ACT_GELU_TANH>()); break;
              case SWIN_WATTN_ACT_SILU: activate(std::integral_constant<int, SWIN_WATTN_ACT_SILU>()); break;
              default: activate(std::integral_constant<int, SWIN_WATTN_ACT_NONE>()); break;
            }
          } else {
            if constexpr (EPI == kEpiGram || EPI == kEpiPoly) {
              if (w.n0 + c0 == row0) {  // the diagonal's slices: both are multiples of 32
#pragma unroll
                for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) + (lane == e ? p.diag : 0.0f));
                if (EPI == kEpiPoly && row < p.M) {
                  const float x = __half2float(reinterpret_cast<const __half*>(at(sr, lane >> 3))[lane & 7]);
                  const float entry = fmaf(of_lane(a, lane), p.alpha, x * p.beta);
                  p.gain[(int64_t)w.b * p.gain_ld + row] = __fdividef(entry, __half2float(__float2half_rn(entry)));
                }
              }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint4 r = make_uint4(0, 0, 0, 0);
              if (aux) r = *at(sr, c);
              const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int e = 8 * c + 2 * q;
                if constexpr (EPI == kEpiGrad16) {
                  const float2 y = __fadd2_rn(pair(e), unpack_bf16(rr[q]));
                  o[4 * c + q] = pack_bf16(y.x, y.y);
                } else if constexpr (EPI == kEpiUpdate) {
                  const float4 f = factor[2 * c + q / 2];
                  const float2 y = __fmul2_rn(pair(e), q % 2 ? make_float2(f.z, f.w) : make_float2(f.x, f.y));
                  if (parts) {
                    o[4 * c + q] = pack_f16(y.x, y.y);
                    const float2 rest = fsub2(y, unpack_f16(o[4 * c + q]));
                    low[4 * c + q] = pack_f16(rest.x, rest.y);
                  } else {
                    o[4 * c + q] = pack_bf16(y.x, y.y);
                  }
                } else {
                  float2 y = __fmul2_rn(pair(e), splat(p.alpha));
                  if constexpr (EPI == kEpiPoly) y = __ffma2_rn(pair(e), splat(p.alpha), __fmul2_rn(unpack_f16(rr[q]), splat(p.beta)));
                  o[4 * c + q] = pack_f16(y.x, y.y);
                }
              }
            }
          }
          tile_free();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            *at(sr, c) = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            if (EPI == kEpiAct && pre) {
              uint32_t z16[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) z16[q] = pack_bf16(pair(8 * c + 2 * q).x, pair(8 * c + 2 * q).y);
              *at(sz + lane * 64, c) = make_uint4(z16[0], z16[1], z16[2], z16[3]);
            }
            if constexpr (EPI == kEpiUpdate)
              if (parts) *at(sz + lane * 64, c) = make_uint4(low[4 * c], low[4 * c + 1], low[4 * c + 2], low[4 * c + 3]);
          }
          if (symmetric(EPI) && mirror) {
#pragma unroll
            for (int e = 0; e < 32; ++e)  // column e becomes row e
              *reinterpret_cast<uint16_t*>(sz + e * 64 + (((lane >> 3) ^ ((e >> 1) & 3)) << 4) + (lane & 7) * 2) =
                  (uint16_t)(e & 1 ? o[e / 2] >> 16 : o[e / 2]);
          }
        }
        if (EPI == kEpiUpdate && p.raw_out != nullptr) {
          __syncwarp();
          const int col = w.n0 + c0 + lane;
          if (col < p.N)
            for (int r = 0; r < 32 && row0 + r < p.M; ++r)
              p.raw_out[((int64_t)w.b * p.M + row0 + r) * p.N + col] = *reinterpret_cast<const __nv_bfloat16*>(
                  so + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
          __syncwarp();  // every lane has read the tile
        } else {
          tc::fence_proxy_async();  // the staging tile to the copy engine
          __syncwarp();
          if (lane == 0) {
            const int batch = EPI == kEpiGrad32 ? w.b * p.n_splits.d + w.split : parts ? 2 * w.b : w.b;
            store_3d(&out_map, w.n0 + c0, row0, batch, smem_u32(so));
            if (parts) store_3d(&out_map, w.n0 + c0, row0, batch + 1, smem_u32(sz));
            if (EPI == kEpiAct && pre) store_3d(&pre_map, w.n0 + c0, row0, w.b, smem_u32(sz));
            if (symmetric(EPI) && mirror) store_3d(&out_map, row0, w.n0 + c0, w.b, smem_u32(sz));
            tc::bulk_commit();
          }
        }
        ++m;
        if (++tile == NB) {
          tile = 0;
          aux_phase ^= 1;
        }
      }
      if (bad) break;
      if constexpr (EPI != kEpiGrad32) release();
    }
    if constexpr (kHasAux) {
      // after a timeout: the loads still in flight land before the CTA leaves
      for (; m < issued; ++m) {
        warp_wait(aux0 + 8 * tile, aux_phase, p.wait_ns);
        if (++tile == NB) {
          tile = 0;
          aux_phase ^= 1;
        }
      }
    }
    if constexpr (CG == 2) cluster_arrive();  // while the last stores are written
    if (lane == 0) tc::bulk_wait_all();
  }
  if constexpr (CG == 2)
    if (warp >= kEW) cluster_arrive();
  if (bad && p.status != nullptr) atomicOr(p.status, 1);

  tc::fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_wait();
  if (warp == kMMA) tmem_dealloc<CG>(tmem);
}

// ---- host side ------------------------------------------------------------------------
//
// In an unnamed namespace: the variables that remember what a device has been asked or told
// belong to one library. (With external linkage they are unique in a process, and the
// fault-injection build, loaded beside the library, would find its kernels' attributes set.)
namespace {

// One GB300: 152 SMs, 76 pairs. The tile choice is made for that and does not ask the
// device, so that workspace sizes depend on the shape alone.
constexpr int kSms = 152;
// Clusters of each size that are resident at once on one GB300 (as cudaOccupancyMaxActiveClusters
// reports them at one CTA per SM: a cluster stays within a group of SMs, and the groups are
// not multiples of every size).
constexpr int kResidentClusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};

// What a launch asks of the current device; read once per device.
struct DeviceInfo {
  int device, smem_max, sms;
};
inline cudaError_t device_info(DeviceInfo* d) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // 0, or SMs * 2^20 + shared memory per block
  cudaError_t e = cudaGetDevice(&d->device);
  if (e != cudaSuccess) return e;
  const int slot = d->device < kDevices ? d->device : -1;
  const int k = slot >= 0 ? known[slot].load(std::memory_order_relaxed) : 0;
  if (k != 0) {
    d->smem_max = k & 0xfffff;
    d->sms = k >> 20;
    return cudaSuccess;
  }
  e = cudaDeviceGetAttribute(&d->smem_max, cudaDevAttrMaxSharedMemoryPerBlockOptin, d->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->device);
  if (e == cudaSuccess && slot >= 0 && d->sms < 2048 && d->smem_max < (1 << 20))
    known[slot].store(d->sms << 20 | d->smem_max, std::memory_order_relaxed);
  return e;
}
// Raise a kernel's dynamic shared memory limit, once per device (64 of them remembered).
inline cudaError_t allow_smem(const void* kern, int bytes, int device, std::atomic<uint64_t>* allowed) {
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (allowed->load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) allowed->fetch_or(bit, std::memory_order_release);
  return e;
}

// A matrix stack [batch, rows, cols], row-major, `ld` elements from row to row.
struct Matrix {
  const void* ptr;
  int64_t rows, cols, ld, batch_stride;
  int parts = 1;  // matrices of the stack to one of the product's batch
};

inline cudaError_t encode_3d(CUtensorMap* map, const Matrix& x, int batch, CUtensorMapDataType type, int elem,
                             int box_cols, int box_rows, CUtensorMapSwizzle swz, CUtensorMapL2promotion l2) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder_fn();
  if (encode == nullptr) return cudaErrorNotSupported;
  const int count = batch * x.parts;
  const cuuint64_t dims[3] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)x.ld * elem, (cuuint64_t)(count > 1 ? x.batch_stride : x.ld) * elem};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(map, type, 3, const_cast<void*>(x.ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swz, l2,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

struct Tiling {
  int cg, NT, splits, chunks, chunks_per_split, n_mt, n_nt;
  bool half;       // only the tiles on and below the diagonal
  int per_matrix;  // tiles that are computed
};

// Estimated time, in SM clocks, of a tiling: rounds of tiles over the SMs (or pairs), each
// the longer of its chunks and its epilogue, plus one epilogue that nothing overlaps and,
// where K is split, the sum of the partial results.
// A chunk of CG * 128 x NT x 64 takes 2 NT clocks of the tensor cores, 200 to issue, and the
// 128 + NT / CG rows of 128 bytes a CTA brings for it (MN-major B comes in blocks of 64) arrive at
// some 53 bytes a clock
// (measured: 24.2 us for 96 chunks of 160 rows, 599 us for 1792 of 256).
inline int b_rows(int NT, int cg, bool bmn) { return bmn ? (NT / cg + 63) / 64 * 64 : NT / cg; }
inline double chunk_clocks(int NT, int cg, bool bmn) {
  return std::max({2.0 * NT, 200.0, 2.4 * (kBM + b_rows(NT, cg, bmn))});
}
// `extra` columns beside a tile's hold the sums over K; where they lie in the other accumulator
// every segment of an fp32 result waits for the last one's epilogue, some 2000 clocks. (Of several
// columns of tiles only the first pays that, which is not charged: 12544 x 1536 x 6144 takes 167 us
// with the sums, 157 us without.)
inline double tiling_cost(const Tiling& t, int64_t M, int64_t N, int batch, bool bmn, bool sums) {
  const int64_t items = (int64_t)t.per_matrix * t.splits * batch;
  const int64_t groups = kSms / t.cg;
  const double rounds = (double)((items + groups - 1) / groups);
  const double epi = 500.0 + 14.0 * t.NT;
  double cost = 5000.0 + rounds * std::max(t.chunks_per_split * chunk_clocks(t.NT, t.cg, bmn), epi) + epi;
  if (sums && t.n_nt == 1 && t.NT + 16 * t.cg > kMaxNT) cost += rounds * 2000.0 * (t.chunks_per_split / kSegChunks);
  // the second, transposed stores and their staging (eight 2048 x 512, all tiles 151 us, half 157
  // us; two 1536 x 6144, 451 and 419 us)
  if (t.half) cost += 2500.0;
  if (t.splits > 1) cost += 4000.0 + (double)(t.splits + 1) * M * N * batch * 4.0 / 3000.0;
  return cost;
}

// The cheapest tiling. `max_splits` > 1 allows K to be split into partial results.
inline Tiling search_tiling(int64_t M, int64_t N, int64_t K, int batch, bool bmn, int max_splits, bool sums, bool sym) {
  Tiling best{};
  double best_cost = -1.0;
  const int chunks = (int)((K + kKC - 1) / kKC);
  for (int cg = 1; cg <= 2; ++cg) {
    for (int nt = kMaxNT; nt >= 32; nt -= 32) {
      Tiling t{};
      t.cg = cg;
      t.NT = nt;
      t.chunks = chunks;
      t.n_mt = (int)((M + cg * kBM - 1) / (cg * kBM));
      t.n_nt = (int)((N + nt - 1) / nt);
      for (int half = 0; half <= (sym ? 1 : 0); ++half) {
        t.half = half != 0;
        t.per_matrix = t.n_mt * t.n_nt;
        if (t.half) {
          t.per_matrix = 0;
          for (int mt = 0; mt < t.n_mt; ++mt) t.per_matrix += lower_tiles(mt, cg * kBM, nt, t.n_nt, FastDiv());
        }
        for (int s = 1; s <= max_splits; ++s) {
          const int per = (chunks + s - 1) / s;
          if (s > 1 && per < 4) break;
          if ((chunks + per - 1) / per != s) continue;  // every split has chunks
          t.splits = s;
          t.chunks_per_split = per;
          const double c = tiling_cost(t, M, N, batch, bmn, sums);
          if (best_cost < 0.0 || c < best_cost) {
            best_cost = c;
            best = t;
          }
        }
      }
    }
  }
  return best;
}

// The same, with the calling thread's last choices remembered by their sizes (a search
// compares some hundred tilings, which is more than a small launch takes).
inline Tiling choose_tiling(int64_t M, int64_t N, int64_t K, int batch, bool bmn, int max_splits, bool sums,
                            bool sym = false) {
  struct Entry {
    int64_t key[8];
    Tiling t;
  };
  constexpr int kEntries = 64;
  thread_local Entry cache[kEntries] = {};
  const int64_t key[8] = {M, N, K, batch, bmn, max_splits, sums, sym};
  uint64_t h = 0;
  for (const int64_t k : key) h = (h ^ (uint64_t)k) * 0x9E3779B97F4A7C15ull;
  Entry& c = cache[h >> 58];
  if (!std::equal(key, key + 8, c.key)) {
    c.t = search_tiling(M, N, K, batch, bmn, max_splits, sums, sym);
    std::copy(key, key + 8, c.key);
  }
  return c.t;
}

// Chunks of K from which K is long.
constexpr int kLongK = 20;

struct Extra {
  const Matrix* aux = nullptr;
  const Matrix* pre = nullptr;
};

template <int CG, bool AMN, bool BMN, int EPI>
cudaError_t launch_tiles(const Tiling& t, Params p, const Matrix& a, const Matrix& b, const Matrix& out, int batch,
                         CUtensorMapDataType in_type, CUtensorMapDataType out_type, const Extra& ex, cudaStream_t st) {
  constexpr int kTile = tile_bytes(EPI);
  constexpr CUtensorMapSwizzle kOutSwz = EPI == kEpiGrad32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  constexpr CUtensorMapL2promotion kL2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  CUtensorMap a_map, b_map, out_map, aux_map, pre_map;
  cudaError_t e = encode_3d(&a_map, a, batch, in_type, 2, kKC, AMN ? 64 : kBM, CU_TENSOR_MAP_SWIZZLE_128B, kL2);
  if (e == cudaSuccess)
    e = encode_3d(&b_map, b, batch, in_type, 2, kKC, BMN ? 64 : t.NT / CG, CU_TENSOR_MAP_SWIZZLE_128B, kL2);
  if (e != cudaSuccess) return e;
  if (p.raw_out == nullptr) {
    e = encode_3d(&out_map, out, EPI == kEpiGrad32 ? t.splits * batch : batch, out_type, EPI == kEpiGrad32 ? 4 : 2, kSC, 32,
                  kOutSwz, CU_TENSOR_MAP_L2_PROMOTION_NONE);
    if (e != cudaSuccess) return e;
  } else {
    out_map = a_map;  // not used
  }
  aux_map = pre_map = a_map;
  p.has_aux = ex.aux != nullptr;
  p.has_pre = ex.pre != nullptr;
  if (p.has_aux) {
    const CUtensorMapDataType aux_type = EPI == kEpiPoly ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    e = encode_3d(&aux_map, *ex.aux, batch, aux_type, 2, kSC, 32, kOutSwz, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    if (e != cudaSuccess) return e;
  }
  if (p.has_pre) {
    e = encode_3d(&pre_map, *ex.pre, batch, out_type, 2, kSC, 32, kOutSwz, CU_TENSOR_MAP_L2_PROMOTION_NONE);
    if (e != cudaSuccess) return e;
  }
  p.NT = t.NT;
  p.n_mt = FastDiv(t.n_mt);
  p.n_nt = FastDiv(t.n_nt);
  p.n_splits = FastDiv(t.splits);
  p.chunks = t.chunks;
  p.chunks_per_split = t.chunks_per_split;
  const int64_t items = (int64_t)t.per_matrix * t.splits * batch;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  p.half = t.half;
  if (t.half) {
    p.n_lower = FastDiv(t.per_matrix);
    p.per_nt = FastDiv(t.NT);
  }
  p.n_items = (int)items;
  p.wait_ns = wait_limit_ns();
  p.fault = fault_site();
  // kind::f16: fp32 accumulator, A and B bf16 (format 1) or fp16 (format 0)
  const uint32_t fmt = in_type == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 0u : (1u << 7) | (1u << 10);
  p.idesc = tc::idesc_bf16(CG * kBM, t.NT, BMN, AMN) ^ fmt;
  p.idesc_ones = tc::idesc_bf16(CG * kBM, 16 * CG, false, AMN) ^ fmt;
  p.stage_bytes = kABytes + b_rows(t.NT, CG, BMN) * 128;
  DeviceInfo di;
  e = device_info(&di);
  if (e != cudaSuccess) return e;
  const int smem_max = di.smem_max, sms = di.sms;
  constexpr int kEW = epi_warps(EPI);
  // the bias of two tiles, or the ones that sum A over K
  constexpr int kSmall = EPI == kEpiAct ? 2 * kMaxNT * 4 : EPI == kEpiGrad32 || EPI == kEpiGrad16 ? 512 : 0;
  const bool long_k = t.chunks_per_split >= kLongK;
  int fixed = 0;
  // a second result's tile, the transposed one, or the smaller part
  const bool second = p.has_pre || t.half || (EPI == kEpiUpdate && !p.to_bf16);
  p.tiles = p.has_aux ? (second || long_k ? 2 : kMaxAuxTiles) : (second || long_k ? 1 : 2);
  for (;; --p.tiles) {  // fewer aux tiles where the ring would not have three stages
    p.warp_bytes = (p.tiles + (second ? 1 : 0)) * kTile;
    fixed = kEW * p.warp_bytes + kSmall + 8 * kNBar + 16;
    p.stages = std::min(kMaxStages, (smem_max - fixed) / p.stage_bytes);
    if (p.stages >= 3 || p.tiles <= 2) break;
  }
  if (p.stages < 2) return cudaErrorInvalidConfiguration;
  p.off_out = p.stages * p.stage_bytes;
  p.off_small = p.off_out + kEW * p.warp_bytes;
  p.off_bar = p.off_small + kSmall;
  // more than half of an SM's shared memory: one CTA per SM, so the tensor memory is free
  const int smem = std::max(120 * 1024, p.off_out + fixed);
  auto kern = product_kernel<CG, AMN, BMN, EPI>;
  static std::atomic<uint64_t> allowed{0};  // devices whose limit has been raised
  e = allow_smem(reinterpret_cast<const void*>(kern), smem_max, di.device, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(CG * std::min<int64_t>(items, sms / CG)));
  cfg.blockDim = dim3(n_threads(EPI));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a_map, b_map, out_map, aux_map, pre_map, p);
}

template <bool AMN, bool BMN, int EPI>
cudaError_t launch_product(const Tiling& t, const Params& p, const Matrix& a, const Matrix& b, const Matrix& out,
                           int batch, CUtensorMapDataType in_type, CUtensorMapDataType out_type, const Extra& ex,
                           cudaStream_t st) {
  return t.cg == 2 ? launch_tiles<2, AMN, BMN, EPI>(t, p, a, b, out, batch, in_type, out_type, ex, st)
                   : launch_tiles<1, AMN, BMN, EPI>(t, p, a, b, out, batch, in_type, out_type, ex, st);
}

}  // namespace
}  // namespace prod
}  // namespace swin
