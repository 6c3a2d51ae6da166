// What the residual sum with its norms (block_norm.cu) and its gradients (block_norm_bwd.cu)
// share: how a row of channels lies in threads, reads and writes of four channels, and the sums
// over a row.
//
// A row is held in registers by a group of threads, `CH` chunks of four consecutive channels each, chunk j of
// thread l at (j * width + l) * 4: a row is read once for all its sums, and its reads are whole lines. Groups
// of 4, 8, 16 or 32 threads lie in a warp and sum by shuffles; a wider row takes a
// block. Two chunks a thread fit the powers of two, three and six 3 * 2^k (96, 192, 384, 768) without idle threads.
#pragma once

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "common.cuh"

namespace swin {
namespace norm {

constexpr int kV = 4;          // channels of a chunk
constexpr int kMaxWarps = 16;  // of a block that holds a row: 512 threads of up to 16 channels

// The shape of a row: the group (0: a block of `threads`) and its chunks.
struct Shape {
  int lanes, chunks, threads, rows_per_block;
};

// Four consecutive channels as two pairs, for packed arithmetic.
struct Four {
  float2 p[2];
};
__device__ __forceinline__ Four zeros() {
  const float2 z = make_float2(0.0f, 0.0f);
  return {{z, z}};
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ Four unpack4(const uint2& w) {
  return {{make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u)),
           make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u))}};
}
__device__ __forceinline__ Four unpack4(const float4& w) { return {{make_float2(w.x, w.y), make_float2(w.z, w.w)}}; }
__device__ __forceinline__ Four load4(const __nv_bfloat16* p) { return unpack4(*reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ Four load4(const float* p) { return unpack4(*reinterpret_cast<const float4*>(p)); }
// Parameters, which may lie at any multiple of four bytes: `vec` where all of them are 16-byte aligned. (One
// value at a time, 12561 x 768 with gate and norm took 33 us instead of 22.)
__device__ __forceinline__ Four load_param4(const float* p, bool vec) {
  if (vec) return load4(p);
  return {{make_float2(__ldg(p), __ldg(p + 1)), make_float2(__ldg(p + 2), __ldg(p + 3))}};
}
inline bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  return true;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const Four& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.p[0].x, v.p[0].y), pack_bf16(v.p[1].x, v.p[1].y));
}
__device__ __forceinline__ void store4(float* p, const Four& v) {
  *reinterpret_cast<float4*>(p) = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
}
__device__ __forceinline__ Four mul(const Four& a, const Four& b) {
  return {{__fmul2_rn(a.p[0], b.p[0]), __fmul2_rn(a.p[1], b.p[1])}};
}
__device__ __forceinline__ Four mul(const Four& a, float b) {
  return {{__fmul2_rn(a.p[0], splat(b)), __fmul2_rn(a.p[1], splat(b))}};
}
__device__ __forceinline__ Four add(const Four& a, const Four& b) {
  return {{__fadd2_rn(a.p[0], b.p[0]), __fadd2_rn(a.p[1], b.p[1])}};
}
__device__ __forceinline__ Four add(const Four& a, float b) {
  return {{__fadd2_rn(a.p[0], splat(b)), __fadd2_rn(a.p[1], splat(b))}};
}
__device__ __forceinline__ Four fma(const Four& a, const Four& b, const Four& c) {
  return {{__ffma2_rn(a.p[0], b.p[0], c.p[0]), __ffma2_rn(a.p[1], b.p[1], c.p[1])}};
}
__device__ __forceinline__ Four fma(const Four& a, float b, const Four& c) {
  return {{__ffma2_rn(a.p[0], splat(b), c.p[0]), __ffma2_rn(a.p[1], splat(b), c.p[1])}};
}

// Sums over a row, the same in every thread of its group. A block adds up its warps' sums in every warp; of two sums
// each half of a warp takes one, 10 exchanges instead of 18, but for kWhole. kEven: its warps are a power of two, of which only
// those that are there are added up. (Gradients of 18816 x 1024, without a norm behind and with one: kWhole 49.3 and 64.7 us,
// kHalves 54.3 and 59.4, kEven 55.3 and 58.3; forward 2500 x 768 with both norms 5.4 and 5.0.)
enum { kWhole, kHalves, kEven };
template <int LANES, int FORM>
struct RowSum {
  float* slots;  // LANES == 0: shared memory, two sets of two slots for each warp, used in turn
  int set = 0;
  // The sum of the warps' sums, which lie `first` apart in `at`: a lane reads one and those a multiple of `first` away are
  // added. The set written before was last read before the barrier of the sum before this one.
  __device__ __forceinline__ float of_warps(const float* at, int first) {
    const int lane = threadIdx.x & 31, n = (int)(blockDim.x >> 5) * first;
    float v;
    if constexpr (FORM == kEven) {
      v = at[lane & (n - 1)];
      for (int o = first; o < n; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else {
      v = (lane & (kMaxWarps * first - 1)) < n ? at[lane & (kMaxWarps * first - 1)] : 0.0f;
#pragma unroll
      for (int o = kMaxWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o * first);
    }
    set ^= 1;
    return v;
  }
  __device__ __forceinline__ float operator()(float v) {
    constexpr int kTop = LANES == 0 ? 16 : LANES / 2;
#pragma unroll
    for (int o = kTop; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (LANES == 0) {
      float* const at = slots + set * 2 * kMaxWarps;
      if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = v;
      __syncthreads();
      v = of_warps(at, 1);
    }
    return v;
  }
  __device__ __forceinline__ float2 operator()(float2 v) {
    if constexpr (LANES == 0 && FORM != kWhole) {
      const bool upper = (threadIdx.x & 16) != 0;
      float a = (upper ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, upper ? v.x : v.y, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      float* const at = slots + set * 2 * kMaxWarps;
      if ((threadIdx.x & 15) == 0) at[threadIdx.x >> 4] = a;
      __syncthreads();
      a = of_warps(at, 2);
      const float b = __shfl_xor_sync(0xffffffffu, a, 1);
      v = (threadIdx.x & 1) != 0 ? make_float2(b, a) : make_float2(a, b);
    } else if constexpr (LANES == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
      float2* const at = reinterpret_cast<float2*>(slots + set * 2 * kMaxWarps);
      const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
      if (lane == 0) at[threadIdx.x >> 5] = v;
      __syncthreads();
      v = (lane & 15) < warps ? at[lane & 15] : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int o = kMaxWarps / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
      set ^= 1;
    } else {
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
    }
    return v;
  }
};

// v <- (v - mean) / sqrt(var + eps), or v / sqrt(mean of v^2 + eps); returns that factor. The mean is
// taken out before the squares are summed, so a mean far above the spread costs nothing. Chunks
// outside the row hold zeros and are left zero.
template <int LANES, int CH, int FORM>
__device__ __forceinline__ float normalise(Four (&v)[CH], const bool (&in)[CH], bool rms, float inv_c, float eps,
                                           RowSum<LANES, FORM>& sum) {
  if (!rms) {
    Four s = v[0];
#pragma unroll
    for (int j = 1; j < CH; ++j) s = add(s, v[j]);
    const float2 t = __fadd2_rn(s.p[0], s.p[1]);
    const float mean = sum(t.x + t.y) * inv_c;
#pragma unroll
    for (int j = 0; j < CH; ++j) v[j] = add(v[j], in[j] ? -mean : 0.0f);
  }
  Four s = mul(v[0], v[0]);
#pragma unroll
  for (int j = 1; j < CH; ++j) s = fma(v[j], v[j], s);
  const float2 t = __fadd2_rn(s.p[0], s.p[1]);
  const float r = rsqrtf(fmaf(sum(t.x + t.y), inv_c, eps));
#pragma unroll
  for (int j = 0; j < CH; ++j) v[j] = mul(v[j], r);
  return r;
}

// The same for two rows at once, with half the rounds of sums.
template <int LANES, int CH, int FORM>
__device__ __forceinline__ float2 normalise_both(Four (&v)[CH], Four (&u)[CH], const bool (&in)[CH], bool rms, float inv_c,
                                                 float eps, RowSum<LANES, FORM>& sum) {
  auto pair_sum = [](const Four& a, const Four& b) {
    const float2 x = __fadd2_rn(a.p[0], a.p[1]), y = __fadd2_rn(b.p[0], b.p[1]);
    return make_float2(x.x + x.y, y.x + y.y);
  };
  if (!rms) {
    Four a = v[0], b = u[0];
#pragma unroll
    for (int j = 1; j < CH; ++j) a = add(a, v[j]), b = add(b, u[j]);
    const float2 mean = sum(pair_sum(a, b));
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      v[j] = add(v[j], in[j] ? -mean.x * inv_c : 0.0f);
      u[j] = add(u[j], in[j] ? -mean.y * inv_c : 0.0f);
    }
  }
  Four a = mul(v[0], v[0]), b = mul(u[0], u[0]);
#pragma unroll
  for (int j = 1; j < CH; ++j) a = fma(v[j], v[j], a), b = fma(u[j], u[j], b);
  const float2 var = sum(pair_sum(a, b));
  const float2 r = make_float2(rsqrtf(fmaf(var.x, inv_c, eps)), rsqrtf(fmaf(var.y, inv_c, eps)));
#pragma unroll
  for (int j = 0; j < CH; ++j) v[j] = mul(v[j], r.x), u[j] = mul(u[j], r.y);
  return r;
}

// ---- rows on their way ----------------------------------------------------------------
//
// A thread's part of the rows to come travels through slots of its own in shared memory by asynchronous copies: no
// thread waits for another, and no register holds a row before its turn. A stage holds one row of each group.

// A chunk as it lies in memory.
template <typename S>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  using T = uint2;
};
template <>
struct Raw<float> {
  using T = float4;
};
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  if constexpr (BYTES == 16)
    cp_async_16(smem_u32(to), from);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(smem_u32(to)), "l"(from), "n"(BYTES) : "memory");
}
constexpr int kMaxSmem = 226 * 1024;  // of the blocks on an SM

// Raise a kernel's shared memory limit (once for each device) and launch it.
template <auto KERN, typename Params>
inline cudaError_t launch_rows(const Params& p, int blocks, int threads, int smem, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  if (smem > 47 * 1024) {  // beside the static part
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if ((allowed.load(std::memory_order_acquire) & bit) == 0) {
      e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      if (e != cudaSuccess) return e;
      allowed.fetch_or(bit, std::memory_order_release);
    }
  }
  return launch_pdl(KERN, dim3(blocks), dim3(threads), smem, st, p);
}

}  // namespace norm
}  // namespace swin
