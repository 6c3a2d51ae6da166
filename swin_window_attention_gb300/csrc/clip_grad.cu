// The norm over all gradients of a model, and their clipping:
//   n = scale |g|,   out = g * scale * min(1, max_norm / (n + eps))
// over any number of fp32 and bf16 tensors of any size and alignment. A plan cuts the tensors into pieces, of which there
// is a list in device memory, and blocks take pieces in turn, so that one launch covers hundreds of tensors of
// all sizes. (With the tensors' addresses as kernel parameters and a search for each piece, whose steps miss the
// constant cache one after the other, 196 M gradients took 225 us.)
// * squares_kernel: a block's sum of squares, one for each block, in the workspace.
// * scale_kernel: every block adds those up in the same order (the same bits on every run),
//   forms the factor, and scales its pieces, from the last one back: what the first launch read
//   last is still in L2.
// Where the factor is 1 and the tensors are scaled in place there is nothing to write.
#include <algorithm>
#include <cfloat>
#include <new>
#include <vector>

#include "clip_grad.cuh"
#include "common.cuh"

namespace swin {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 4 * 152;

using Piece = ClipPiece;
// One of the list, as two 16-byte reads.
__device__ __forceinline__ Piece piece_at(const Piece* list, uint32_t i) {
  union {
    uint4 w[2];
    Piece p;
  } u;
  u.w[0] = __ldg(reinterpret_cast<const uint4*>(list + i));
  u.w[1] = __ldg(reinterpret_cast<const uint4*>(list + i) + 1);
  return u.p;
}

// Conversions and products that keep subnormal numbers (the library is built to flush them).
__device__ __forceinline__ double to_double(float v) {
  double r;
  asm("cvt.f64.f32 %0, %1;\n" : "=d"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float to_float(double v) {
  float r;
  asm("cvt.rn.f32.f64 %0, %1;\n" : "=f"(r) : "d"(v));
  return r;
}
__device__ __forceinline__ float mul_exact(float a, float b) {
  float r;
  asm("mul.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// 16 bytes as fp32 values.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[16 / sizeof(T)]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(in[i]);
    } else {
      v[2 * i] = __uint_as_float(in[i] << 16);
      v[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
    }
  }
}

// Elements before the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int len) {
  return min(len, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T));
}

constexpr int kLoads = 4;  // 16-byte loads of a thread in flight
// A 16-byte read that L2 may drop at once, or keep.
__device__ __forceinline__ uint4 read16(const uint4* p, bool keep) { return keep ? *p : __ldcs(p); }

// A sum of squares: hi + lo in two fp32 parts (48 bits), and beside it `wide`, of those that fp32 does not hold. The GPU
// adds two 64-bit numbers in the time of 64 fp32 additions: with 64-bit sums throughout, 1.2 M gradients took 21 us
// and 393 MB of them were read at 5.8 TB/s.
struct Sum {
  float hi, lo;
  double wide;
};
// hi + lo + v in two parts (Knuth's two-sum, then the parts brought in order).
__device__ __forceinline__ void add(Sum& s, float v) {
  const float t = __fadd_rn(s.hi, v), b = __fsub_rn(t, s.hi);
  const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(v, b));
  s.lo = __fadd_rn(s.lo, e);
  s.hi = t;
}
__device__ __forceinline__ void add(Sum& s, const Sum& o) {
  add(s, o.hi);
  s.lo = __fadd_rn(s.lo, o.lo);
}

// The squares of up to 64 bytes a thread are summed in fp32. That holds where the sum comes out between these bounds: no
// square has overflowed, and those lost (below 2^-126 each) are below its rounding. Else (tiny, huge or no values,
// NaN) they are summed again in 64 bits.
__device__ __forceinline__ bool holds(float s) { return s >= 0x1p-94f && s <= 0x1p96f; }

template <typename T>
__device__ void squares(const T* p, int len, bool keep, Sum& sum) {
  constexpr int kPer = 16 / sizeof(T);
  const int head = head_of(p, len), vecs = (len - head) / kPer, tail = head + vecs * kPer;
  auto one = [&](const T* q) {
    const float v = value(q), s = v * v;
    if (holds(s))
      add(sum, s);
    else
      sum.wide += to_double(v) * to_double(v);
  };
  if ((int)threadIdx.x < head) one(p + threadIdx.x);
  if (tail + (int)threadIdx.x < len) one(p + tail + threadIdx.x);
  const uint4* body = reinterpret_cast<const uint4*>(p + head);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kThreads * kLoads) {
    uint4 w[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) w[k] = i0 + k * kThreads < vecs ? read16(body + i0 + k * kThreads, keep) : make_uint4(0, 0, 0, 0);
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      float v[kPer];
      unpack<T>(w[k], v);
#pragma unroll
      for (int e = 0; e < kPer; e += 2) s = __ffma2_rn(make_float2(v[e], v[e + 1]), make_float2(v[e], v[e + 1]), s);
    }
    const float all = s.x + s.y;
    if (holds(all)) {
      add(sum, all);
    } else {
      uint32_t bits = 0;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) bits |= w[k].x | w[k].y | w[k].z | w[k].w;
      if ((bits & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) == 0) continue;  // zeros
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        float v[kPer];
        unpack<T>(w[k], v);
#pragma unroll 1
        for (int e = 0; e < kPer; ++e) sum.wide = fma(to_double(v[e]), to_double(v[e]), sum.wide);
      }
    }
  }
}

// Whether there are squares that fp32 does not hold (NaN among them). Of the bits: a comparison in 64 bits takes the time
// of 64 others.
__device__ __forceinline__ bool has_wide(const Sum& s) { return (__double2hiint(s.wide) | __double2loint(s.wide)) != 0; }

template <int N>
__device__ __forceinline__ void warp_sum(Sum& v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    Sum u;
    u.hi = __shfl_xor_sync(0xffffffffu, v.hi, o);
    u.lo = __shfl_xor_sync(0xffffffffu, v.lo, o);
    add(v, u);
  }
  if (__any_sync(0xffffffffu, has_wide(v))) {
#pragma unroll 1
    for (int o = N / 2; o > 0; o >>= 1) v.wide += __shfl_xor_sync(0xffffffffu, v.wide, o);
  }
}
// The sum over the block, in the first warp.
__device__ __forceinline__ Sum block_sum(Sum v) {
  constexpr int kWarps = kThreads / 32;
  __shared__ Sum warps[kWarps];
  warp_sum<32>(v);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = warps[threadIdx.x % kWarps];
    warp_sum<kWarps>(v);
  }
  return v;
}

__global__ void __launch_bounds__(kThreads)
    squares_kernel(const Piece* __restrict__ list, uint32_t pieces, uint32_t keep_from, Sum* partial) {
  pdl_launch_dependents();
  Piece next = piece_at(list, blockIdx.x);  // (the list was written when the plan was made)
  pdl_wait();
  Sum sum{0.0f, 0.0f, 0.0};
  for (uint32_t i = blockIdx.x; i < pieces; i += gridDim.x) {
    const Piece p = next;
    if (i + gridDim.x < pieces) next = piece_at(list, i + gridDim.x);
    const bool keep = i >= keep_from;
    if (p.bf16)
      squares(static_cast<const __nv_bfloat16*>(p.in), p.len, keep, sum);
    else
      squares(static_cast<const float*>(p.in), p.len, keep, sum);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void scale_one(const T* in, T* out, float first, float factor) {
  const float v = mul_exact(mul_exact(value(in), first), factor);
  if constexpr (sizeof(T) == 4)
    *out = v;
  else
    *out = __float2bfloat16_rn(v);
}

template <typename T>
__device__ void scale_piece(const T* in, T* out, int len, float first, float factor) {
  constexpr int kPer = 16 / sizeof(T);
  if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
    for (int i = threadIdx.x; i < len; i += kThreads) scale_one(in + i, out + i, first, factor);
    return;
  }
  const int head = head_of(in, len), vecs = (len - head) / kPer, tail = head + vecs * kPer;
  if ((int)threadIdx.x < head) scale_one(in + threadIdx.x, out + threadIdx.x, first, factor);
  if (tail + (int)threadIdx.x < len) scale_one(in + tail + threadIdx.x, out + tail + threadIdx.x, first, factor);
  const uint4* from = reinterpret_cast<const uint4*>(in + head);
  uint4* to = reinterpret_cast<uint4*>(out + head);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kThreads * kLoads) {
    uint4 w[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (i0 + k * kThreads < vecs) w[k] = __ldcs(from + i0 + k * kThreads);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      if (i0 + k * kThreads >= vecs) break;
      float v[kPer];
      unpack<T>(w[k], v);
      if (first != 1.0f) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = mul_exact(v[e], first);
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] = mul_exact(v[e], factor);
      uint4 o;
      if constexpr (sizeof(T) == 4)
        o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      else
        o = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      __stcs(to + i0 + k * kThreads, o);
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    scale_kernel(const Piece* __restrict__ list, uint32_t pieces, const Sum* partial, int n_partial, float max_norm,
                 float scale, float eps, bool in_place, float* norm) {
  pdl_launch_dependents();
  Piece next{};
  if (blockIdx.x < pieces) next = piece_at(list, pieces - 1 - blockIdx.x);
  pdl_wait();
  Sum sum{0.0f, 0.0f, 0.0};
  for (int i = threadIdx.x; i < n_partial; i += kThreads) {
    const float4 raw = __ldcg(reinterpret_cast<const float4*>(partial) + i);
    const Sum o = *reinterpret_cast<const Sum*>(&raw);
    add(sum, o);
    if (has_wide(o)) sum.wide += o.wide;
  }
  sum = block_sum(sum);
  __shared__ float shared_first, shared_factor;
  if (threadIdx.x == 0) {
    // the root of the fp32 sum, or where there is more, that in 64 bits
    float n = scale * __fsqrt_rn(sum.hi + sum.lo);
    if (has_wide(sum)) n = (float)((double)scale * sqrt((double)sum.hi + (double)sum.lo + sum.wide));
    const float c = __fdiv_rn(max_norm, n + eps);
    float first = 1.0f, factor = scale * (c > 1.0f ? 1.0f : c);  // NaN stays NaN
    // Where the norm or the factor leaves fp32's normal range, both in 64 bits, and a factor below it in two: the values
    // times 2^-126, exactly but for those whose results are subnormal, and that times the rest.
    if (!(n >= FLT_MIN && n + eps <= FLT_MAX && factor >= FLT_MIN)) {
      const double root = sqrt((double)sum.hi + (double)sum.lo + sum.wide), wide = to_double(scale) * root;
      const double d = to_double(max_norm) / (wide + to_double(eps)), f = to_double(scale) * (d > 1.0 ? 1.0 : d);
      n = to_float(wide);
      if (f < 0x1p-126 && f > 0.0) first = 0x1p-126f;
      factor = to_float(first == 1.0f ? f : f * 0x1p126);
    }
    if (norm != nullptr && blockIdx.x == 0) *norm = n;
    shared_first = first;
    shared_factor = factor;
  }
  __syncthreads();
  const float first = shared_first, factor = shared_factor;
  if (in_place && first == 1.0f && factor == 1.0f) return;
  for (uint32_t i = blockIdx.x; i < pieces; i += gridDim.x) {
    const Piece p = next;
    if (i + gridDim.x < pieces) next = piece_at(list, pieces - 1 - i - gridDim.x);
    if (p.bf16)
      scale_piece(static_cast<const __nv_bfloat16*>(p.in), static_cast<__nv_bfloat16*>(p.out), p.len, first, factor);
    else
      scale_piece(static_cast<const float*>(p.in), static_cast<float*>(p.out), p.len, first, factor);
  }
}

// Elements of a piece: some four pieces for each block that fits, of 2048 to 16384 elements (a thread's loads are then 16
// bytes times kLoads and a few times that), and more where the list would be longer than 2 MB.
int64_t piece_of_total(int64_t total) {
  int64_t piece = 2048;
  while (piece < 16384 && total / piece > 4 * kMaxBlocks) piece *= 2;
  while (total / piece > 65536) piece *= 2;
  return piece;
}

// What the first launch leaves in L2 for the second: half of it. All other reads and the writes of the second may be dropped
// at once. (392 MB in, as much out: 192 us without these hints, 182 with the reads' of the first launch, 179 with all.)
constexpr int64_t kKeepBytes = 64 << 20;

}  // namespace

size_t clip_piece_count(const int64_t* sizes, int count) {
  int64_t total = 0, n = 0;
  for (int i = 0; i < count; ++i) total += sizes[i];
  const int64_t piece = piece_of_total(total);
  for (int i = 0; i < count; ++i) n += (sizes[i] + piece - 1) / piece;
  return (size_t)n;
}

// The list of a plan's pieces (may throw bad_alloc).
void clip_pieces(const void* const* in, void* const* out, const int64_t* sizes, const int* dtypes, int count,
                 std::vector<ClipPiece>* list, ClipShape* shape) {
  int64_t total = 0, kept = 0;
  shape->in_place = true;
  for (int i = 0; i < count; ++i) {
    total += sizes[i];
    if (sizes[i] > 0 && in[i] != out[i]) shape->in_place = false;
  }
  const int64_t piece = piece_of_total(total);
  for (int i = 0; i < count; ++i) {
    const bool bf16 = dtypes[i] == SWIN_WATTN_BF16;
    for (int64_t at = 0; at < sizes[i]; at += piece) {
      const int64_t bytes = at * (bf16 ? 2 : 4);
      list->push_back({static_cast<const char*>(in[i]) + bytes, static_cast<char*>(out[i]) + bytes,
                       (int)std::min(piece, sizes[i] - at), bf16 ? 1 : 0, 0, 0});
    }
  }
  shape->pieces = (uint32_t)list->size();
  shape->keep_from = shape->pieces;
  while (shape->keep_from > 0 && kept < kKeepBytes) {
    const ClipPiece& p = (*list)[--shape->keep_from];
    kept += (int64_t)p.len * (p.bf16 ? 2 : 4);
  }
}

size_t clip_workspace_bytes() { return kMaxBlocks * sizeof(Sum); }
int clip_launches(const ClipShape& s) { return s.pieces == 0 ? 1 : 2; }

cudaError_t clip_launch(const ClipPiece* list, const ClipShape& s, float max_norm, float scale, float eps, float* norm,
                        void* workspace, cudaStream_t st) {
  Sum* partial = static_cast<Sum*>(workspace);
  const int blocks = (int)std::min<uint32_t>(s.pieces, kMaxBlocks);
  if (blocks > 0) {
    const cudaError_t e = launch_pdl(squares_kernel, dim3(blocks), dim3(kThreads), 0, st, list, s.pieces, s.keep_from, partial);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(scale_kernel, dim3(std::max(1, blocks)), dim3(kThreads), 0, st, list, s.pieces, (const Sum*)partial, blocks,
                    max_norm, scale, eps, s.in_place, norm);
}

}  // namespace swin
