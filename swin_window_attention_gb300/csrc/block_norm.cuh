// What the residual sum with its norms (block_norm.cu) and its gradients (block_norm_bwd.cu)
// share: how a row of channels lies in threads, reads and writes of eight channels, and the sums
// over a row.
//
// A row is held in registers by a group of threads, `CH` chunks of eight consecutive channels (16
// bytes in bf16) each, chunk j of thread l at (j * width + l) * 8, so that every read is whole
// and a row is read once for all its sums. Groups of 4, 8, 16 or 32 threads lie in a warp and sum by
// shuffles; a row of more than 96 chunks takes a block.
#pragma once

#include "common.cuh"

namespace swin {
namespace norm {

constexpr int kMaxC = 8192;
constexpr int kThreads = 256;  // of a block of groups that lie in warps

// The shape for C channels: the group (0: a block of `threads`) and its chunks, of the least
// capacity. Three chunks a thread fit widths of 3 * 2^k (96, 192, 384, 768) without idle threads.
struct Shape {
  int lanes, chunks, threads, rows_per_block;
};
inline Shape shape_of(int C) {
  const int n = C / 8;
  for (int lanes = 4; lanes <= 32; lanes *= 2)
    for (int ch = 2; ch <= 3; ++ch)
      if (n <= lanes * ch) return {lanes, ch, kThreads, kThreads / lanes};
  return {0, 2, ((n + 1) / 2 + 31) / 32 * 32, 1};
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(in[i] << 16);
    v[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// The parameters, which lie at any multiple of four bytes.
__device__ __forceinline__ void load_param8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __ldg(p + e);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sums over a row, the same in every thread of its group.
template <int LANES>
struct RowSum {
  float2* slots;  // LANES == 0: shared memory, two sets of a slot for each warp, used in turn
  int set = 0;
  __device__ __forceinline__ float2 operator()(float2 v) {
    constexpr int kTop = LANES == 0 ? 16 : LANES / 2;
#pragma unroll
    for (int o = kTop; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (LANES == 0) {
      const int warps = blockDim.x >> 5;
      // the set written here was last read before the barrier of the sum before this one
      if ((threadIdx.x & 31) == 0) slots[set * 16 + (threadIdx.x >> 5)] = v;
      __syncthreads();
      v = make_float2(0.0f, 0.0f);
      for (int w = 0; w < warps; ++w) {
        const float2 a = slots[set * 16 + w];
        v.x += a.x;
        v.y += a.y;
      }
      set ^= 1;
    }
    return v;
  }
  __device__ __forceinline__ float operator()(float v) {
    constexpr int kTop = LANES == 0 ? 16 : LANES / 2;
#pragma unroll
    for (int o = kTop; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (LANES == 0) {
      const int warps = blockDim.x >> 5;
      if ((threadIdx.x & 31) == 0) slots[set * 16 + (threadIdx.x >> 5)].x = v;
      __syncthreads();
      v = 0.0f;
      for (int w = 0; w < warps; ++w) v += slots[set * 16 + w].x;
      set ^= 1;
    }
    return v;
  }
};

// v <- (v - mean) / sqrt(var + eps), or v / sqrt(mean of v^2 + eps); returns that factor. The mean is
// taken out before the squares are summed, so a mean far above the spread costs nothing. Chunks
// outside the row hold zeros and are left zero.
template <int LANES, int CH>
__device__ __forceinline__ float normalise(float (&v)[CH][8], const bool (&in)[CH], bool rms, float inv_c, float eps,
                                           RowSum<LANES>& sum) {
  float s = 0.0f;
  if (!rms) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[j][e];
    const float mean = sum(s) * inv_c;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = in[j] ? v[j][e] - mean : 0.0f;
  }
  s = 0.0f;
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
  const float r = rsqrtf(fmaf(sum(s), inv_c, eps));
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] *= r;
  return r;
}

}  // namespace norm
}  // namespace swin
