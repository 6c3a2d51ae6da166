// Microscaled 4-bit operands (fp4.cuh): quantisation and back.
//   NVFP4: s = E4M3(amax / 6 / ts), q = E2M1(x / (s ts)); ts given, or the smallest power of two with
//          max |x| <= 6 * 448 ts
//   MXFP4: s = 2^(floor(log2 amax) - 2), q = E2M1(x / s), values beyond 6 s cut to 6 s
// amax over a block; roundings to nearest, ties to even. A power of two as ts makes every border
// between two roundings exact in fp32 and every decoded value exact in bf16. A NaN or an infinity
// makes its block's scale NaN, so the whole block reads back as NaN, and counts nowhere else.
//
// A thread takes 16 elements of a row (two threads share a block of MXFP4), so that a warp reads
// 1 KB of a bf16 row and writes 256 bytes; four or eight neighbours put their scales in one word. It does
// so for the four rows r, r + 32, r + 64, r + 96 of 128, whose scales lie side by side: 16 bytes are written or
// read at once (a word a row, 12561 x 6144 NVFP4 took 48 us to quantise and 63 to read back).
// Bound by memory: 2 + 0.56 bytes an element from bf16.
#include <algorithm>

#include "common.cuh"
#include "fp4_quantize.cuh"

namespace swin {

namespace {

using namespace fp4;

constexpr int kThreads = 256;
constexpr int kAmaxBlocks = 2 * 152, kAmaxLoads = 4;
// Of a thread's four rows, how many are on their way at a time: 128 bytes.
template <typename T>
constexpr int kRows = 8 / (int)sizeof(T);

// The smallest power of two of which amax is at most 2688 = 1.3125 * 2^11 times, not below 2^-90 (so
// that no scale or quotient is subnormal).
__device__ __forceinline__ float tensor_scale_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 11 + ((b & 0x7fffffu) > 0x280000u ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 127 - 90) << 23);
}

// The largest finite magnitude of x, for each block of threads.
template <typename T>
__global__ void __launch_bounds__(kThreads) amax_kernel(const T* __restrict__ x, int64_t n16, float* partial) {
  __shared__ float warps[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  float m = 0.0f;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < n16; i0 += step * kAmaxLoads) {
    Raw16<T> r[kAmaxLoads];
#pragma unroll
    for (int k = 0; k < kAmaxLoads; ++k) r[k] = load16(x + min(i0 + k * step, n16 - 1) * 16);
#pragma unroll
    for (int k = 0; k < kAmaxLoads; ++k) {
      const uint32_t bits = amax_bits(r[k]);
      if (bits < kInfinity) {
        m = fmaxf(m, __uint_as_float(bits));
      } else {
        float2 v[8];
        unpack16(r[k], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (fabsf(v[e].x) < __uint_as_float(kInfinity)) m = fmaxf(m, fabsf(v[e].x));
          if (fabsf(v[e].y) < __uint_as_float(kInfinity)) m = fmaxf(m, fabsf(v[e].y));
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, warps[w]);
    partial[blockIdx.x] = m;
  }
}

struct QuantizeParams {
  const void* x;
  uint8_t *codes, *scales;
  float* tensor_scale;
  const float* partial;  // of amax_kernel, or null where the tensor's scale is given
  int n_partial;
  int rows, K, tiles;    // scale tiles along a row
  int width;             // threads a row (a power of two)
};

// FORMAT 0: NVFP4, 1: MXFP4. `width` threads to a row and its three companions, kThreads / width of such fours a block of
// threads, from the last rows back: what amax_kernel read last is still in L2.
template <typename T, int FORMAT>
__global__ void __launch_bounds__(kThreads, 4) quantize_kernel(const QuantizeParams p) {
  constexpr int kUnits = FORMAT == 0 ? 4 : 8;  // threads to a word of four scales
  pdl_launch_dependents();
  pdl_wait();
  float ts = 1.0f;
  if constexpr (FORMAT == 0) {
    if (p.partial != nullptr) {
      __shared__ float warps[kThreads / 32];
      float m = 0.0f;
      for (int i = threadIdx.x; i < p.n_partial; i += kThreads) m = fmaxf(m, __ldcg(p.partial + i));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, warps[w]);
      ts = tensor_scale_of(m);
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.tensor_scale = ts;
    } else {
      ts = *p.tensor_scale;
    }
  }
  [[maybe_unused]] const float r_ts = reciprocal(ts);
  const int per = kThreads / p.width;
  const int64_t four = (int64_t)(gridDim.x - 1 - blockIdx.x) * per + threadIdx.x / p.width;
  const int64_t row0 = (four >> 5) * 128 + (four & 31);
  if ((four >> 5) * 128 >= p.rows) return;  // (of no rows only the tensor's scale is written)
  const int units = p.tiles * kUnits, used = p.K / 16;
  // (a whole word's threads are in the loops or out of them together: width and units are multiples of kUnits, and
  // the shuffles name their own lanes)
  const unsigned lane = threadIdx.x & 31, peers = ((1u << kUnits) - 1) << (lane & ~(kUnits - 1));
  for (int u = blockIdx.y * p.width + threadIdx.x % p.width; u < units; u += gridDim.y * p.width) {
    uint32_t words[4];
#pragma unroll
    for (int k0 = 0; k0 < 4; k0 += kRows<T>) {
      Raw16<T> raw[kRows<T>];
#pragma unroll
      for (int k = 0; k < kRows<T>; ++k) {
        const int64_t row = row0 + 32 * (k0 + k);
        if (row < p.rows && u < used) raw[k] = load16(static_cast<const T*>(p.x) + row * p.K + u * 16);
      }
#pragma unroll
      for (int k = 0; k < kRows<T>; ++k) {
        const int64_t row = row0 + 32 * (k0 + k);
        uint32_t scale = 0;
        if (row < p.rows && u < used) {
          // (used is even, so both threads of a block of MXFP4 are here)
          const uint2 codes = quantize16<FORMAT>(raw[k], ts, r_ts, 3u << (lane & ~1), scale);
          *reinterpret_cast<uint2*>(p.codes + row * (p.K / 2) + u * 8) = codes;
        }
        const int j = FORMAT == 0 ? lane & 3 : (lane >> 1) & 3;
        uint32_t word = scale << (8 * j);
#pragma unroll
        for (int o = FORMAT == 0 ? 1 : 2; o < kUnits; o <<= 1) word |= __shfl_xor_sync(peers, word, o);
        words[k0 + k] = word;
      }
    }
    if ((lane & (kUnits - 1)) == 0)
      *reinterpret_cast<uint4*>(p.scales + scale_word(row0, u / kUnits, p.tiles)) = make_uint4(words[0], words[1], words[2], words[3]);
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2 (&v)[4]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
}
__device__ __forceinline__ void store8(float* p, const float2 (&v)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}

// Eight codes of a thread, so that a warp's 16-byte stores of bf16 follow one another, of four rows as above.
template <typename T, int FORMAT>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const float* __restrict__ tensor_scale, T* __restrict__ out, int rows, int K, int tiles, int width) {
  pdl_launch_dependents();
  pdl_wait();
  const float ts = FORMAT == 0 ? *tensor_scale : 1.0f;
  const int64_t four = (int64_t)blockIdx.x * (kThreads / width) + threadIdx.x / width;
  const int64_t row0 = (four >> 5) * 128 + (four & 31);
  if (row0 >= rows) return;
  const int units = K / 8;
  for (int u0 = 2 * blockIdx.y * width + threadIdx.x % width; u0 < units; u0 += 2 * gridDim.y * width) {
    // two rounds of four rows on their way
    uint4 w[2];
    uint32_t c[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int u = min(u0 + i * width, units - 1), block = FORMAT == 0 ? u >> 1 : u >> 2;
      w[i] = *reinterpret_cast<const uint4*>(scales + scale_word(row0, block >> 2, tiles));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t row = min(row0 + 32 * k, (int64_t)rows - 1);
        c[i][k] = *reinterpret_cast<const uint32_t*>(codes + row * (K / 2) + u * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int u = u0 + i * width, block = FORMAT == 0 ? u >> 1 : u >> 2;
      const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      if (u >= units) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t row = row0 + 32 * k;
        if (row >= rows) break;
        uint32_t h[4];
        of_e2m1x8(c[i][k], h);
        const uint32_t b = words[k] >> (8 * (block & 3)) & 0xff;
        const float s = FORMAT == 0 ? of_e4m3(b) * ts : of_e8m0(b);
        float2 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
          v[e] = FORMAT == 0 ? __fmul2_rn(q, make_float2(s, s)) : make_float2(mul_exact(q.x, s), mul_exact(q.y, s));
        }
        store8(out + row * K + u * 8, v);
      }
    }
  }
}

// Threads a row (and its companions): the power of two, eight to 128, that leaves the fewest idle in its last block, the
// largest of such. (Every block then does one round: with blocks that walked whole rows, 12561 x 6144 MXFP4 took as
// long, 2001 x 8192 15 us instead of 10.)
int width_of(int units) {
  int best = 8;
  for (int w = 8; w <= 128; w *= 2)
    if ((units + w - 1) / w * w <= (units + best - 1) / best * best) best = w;
  return best;
}

int amax_blocks(int64_t n16) { return (int)std::min<int64_t>(kAmaxBlocks, (n16 + kThreads - 1) / kThreads); }

}  // namespace

size_t fp4_workspace_bytes() { return kAmaxBlocks * sizeof(float); }

cudaError_t fp4_quantize_launch(const void* x, void* codes, void* scales, float* tensor_scale, int rows, int K, int format,
                                int dtype, bool scale_given, void* workspace, cudaStream_t st) {
  QuantizeParams p{};
  p.x = x;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.tensor_scale = tensor_scale;
  p.rows = rows;
  p.K = K;
  p.tiles = k_tiles(K, format);
  p.width = width_of(p.tiles * (format == 0 ? 4 : 8));
  const bool f32 = dtype == SWIN_WATTN_FP32;
  if (format == 0 && !scale_given) {
    const int64_t n16 = (int64_t)rows * (K / 16);
    p.partial = static_cast<float*>(workspace);
    p.n_partial = amax_blocks(n16);
    const dim3 grid(p.n_partial), block(kThreads);
    const cudaError_t e =
        rows == 0 ? cudaSuccess
        : f32 ? launch_pdl(amax_kernel<float>, grid, block, 0, st, static_cast<const float*>(x), n16, static_cast<float*>(workspace))
            : launch_pdl(amax_kernel<__nv_bfloat16>, grid, block, 0, st, static_cast<const __nv_bfloat16*>(x), n16,
                         static_cast<float*>(workspace));
    if (e != cudaSuccess) return e;
  }
  const int per = kThreads / p.width;  // divides 32
  const dim3 grid((unsigned)std::max<int64_t>(1, ((int64_t)rows + 127) / 128 * 32 / per), (p.tiles * (format == 0 ? 4 : 8) + p.width - 1) / p.width), block(kThreads);
  if (format == 0)
    return f32 ? launch_pdl(quantize_kernel<float, 0>, grid, block, 0, st, p)
               : launch_pdl(quantize_kernel<__nv_bfloat16, 0>, grid, block, 0, st, p);
  return f32 ? launch_pdl(quantize_kernel<float, 1>, grid, block, 0, st, p)
             : launch_pdl(quantize_kernel<__nv_bfloat16, 1>, grid, block, 0, st, p);
}

cudaError_t fp4_dequantize_launch(const void* codes, const void* scales, const float* tensor_scale, void* out, int rows,
                                  int K, int format, int dtype, cudaStream_t st) {
  const int tiles = k_tiles(K, format), width = width_of((K / 8 + 1) / 2), per = kThreads / width;
  const dim3 grid((unsigned)(((int64_t)rows + 127) / 128 * 32 / per), (K / 8 + 2 * width - 1) / (2 * width)), block(kThreads);
  auto go = [&](auto kern, auto* to) {
    return launch_pdl(kern, grid, block, 0, st, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                      tensor_scale, to, rows, K, tiles, width);
  };
  if (dtype == SWIN_WATTN_FP32) {
    float* to = static_cast<float*>(out);
    return format == 0 ? go(dequantize_kernel<float, 0>, to) : go(dequantize_kernel<float, 1>, to);
  }
  __nv_bfloat16* to = static_cast<__nv_bfloat16*>(out);
  return format == 0 ? go(dequantize_kernel<__nv_bfloat16, 0>, to) : go(dequantize_kernel<__nv_bfloat16, 1>, to);
}

}  // namespace swin
