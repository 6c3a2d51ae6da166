// Microscaled 4-bit operands (fp4.cuh): quantisation and back.
//   NVFP4: s = E4M3(amax / 6 / ts), q = E2M1(x / (s ts)); ts given, or the smallest power of two with
//          max |x| <= 6 * 448 ts
//   MXFP4: s = 2^(floor(log2 amax) - 2), q = E2M1(x / s), values beyond 6 s cut to 6 s
// amax over a block; roundings to nearest, ties to even. A power of two as ts makes every border
// between two roundings exact in fp32 and every decoded value exact in bf16. A NaN or an infinity
// makes its block's scale NaN, so the whole block reads back as NaN, and counts nowhere else.
//
// A thread takes 16 elements of a row (two threads share a block of MXFP4), so that a warp reads
// 1 KB of a bf16 row and writes 256 bytes; four or eight neighbours put their scales in one word.
// Bound by memory: 2 + 0.56 bytes an element from bf16.
#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"

namespace swin {

namespace {

using namespace fp4;

constexpr int kThreads = 256;
constexpr int kAmaxBlocks = 2 * 152;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Products that keep subnormals (the library is built to flush them).
__device__ __forceinline__ float mul_exact(float a, float b) {
  float r;
  asm("mul.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Eight values to eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xff;
}
// An E4M3 of no sign: (8 + m) 2^(e - 10), or m 2^-9 where e is 0.
__device__ __forceinline__ float of_e4m3(uint32_t b) {
  if (b == 0x7f) return __uint_as_float(0x7fc00000u);
  const uint32_t e = b >> 3, m = b & 7;
  return e == 0 ? (float)m * 0x1p-9f : __uint_as_float((e + 120) << 23 | m << 20);
}
// 2^(b - 127); 0xff is NaN.
__device__ __forceinline__ float of_e8m0(uint32_t b) {
  return __uint_as_float(b == 0xff ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
}

__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(in[i] << 16);
    v[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[16]) {
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  unpack8(a, v);
  unpack8(b, v + 8);
}
__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
  }
}

// The smallest power of two of which amax is at most 2688 = 1.3125 * 2^11 times, not below 2^-90 (so
// that no scale or quotient is subnormal).
__device__ __forceinline__ float tensor_scale_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 11 + ((b & 0x7fffffu) > 0x280000u ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 127 - 90) << 23);
}

// Codes of 16 values x of an NVFP4 block: x / d, correctly rounded, from the rounded reciprocal r of d by
// one correction of the quotient (Markstein, 1990: the remainder of the product is exact in an fma), so
// that ties are met as a division would.
__device__ __forceinline__ uint2 codes_of_quotient(const float (&x)[16], float d, float r) {
  float q[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float q0 = x[e] * r;
    q[e] = fmaf(fmaf(-q0, d, x[e]), r, q0);
  }
  return make_uint2(to_e2m1x8(q), to_e2m1x8(q + 8));
}

// The largest finite magnitude of x, for each block of threads.
template <typename T>
__global__ void __launch_bounds__(kThreads) amax_kernel(const T* __restrict__ x, int64_t n16, float* partial) {
  __shared__ float warps[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  float m = 0.0f;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n16; i += (int64_t)gridDim.x * kThreads) {
    float v[16];
    load16(x + i * 16, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float a = fabsf(v[e]);
      m = a > m && a < __uint_as_float(0x7f800000u) ? a : m;
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

// FORMAT 0: NVFP4, 1: MXFP4. `width` threads a row, kThreads / width rows a block of threads, from the last rows
// back: what amax_kernel read last is still in L2.
template <typename T, int FORMAT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantizeParams p) {
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
      if (blockIdx.x == 0 && threadIdx.x == 0) *p.tensor_scale = ts;
    } else {
      ts = *p.tensor_scale;
    }
  }
  const int64_t row = (int64_t)(gridDim.x - 1 - blockIdx.x) * (kThreads / p.width) + threadIdx.x / p.width;
  const int units = p.tiles * kUnits, used = p.K / 16;
  // (a whole word's threads are in the loop or out of it together: width and units are multiples of kUnits, and
  // the shuffles name their own lanes)
  const unsigned lane = threadIdx.x & 31, peers = ((1u << kUnits) - 1) << (lane & ~(kUnits - 1));
  if (row >= (p.rows + 127) / 128 * (int64_t)128) return;
  for (int u = threadIdx.x % p.width; u < units; u += p.width) {
    uint32_t scale = 0;
    if (row < p.rows && u < used) {
      float v[16];
      load16(static_cast<const T*>(p.x) + row * p.K + u * 16, v);
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) amax = max_nan(amax, fabsf(v[e]));
      uint2 codes = make_uint2(0, 0);
      if constexpr (FORMAT == 0) {
        const float ratio = __fdiv_rn(__fdiv_rn(amax, 6.0f), ts);
        scale = amax < __uint_as_float(0x7f800000u) ? to_e4m3(ratio) : 0x7f;
        const float s = of_e4m3(scale), d = s * ts;
        if (s > 0.0f) {
          if (ratio > 448.0f) {  // a given scale that is too small: the correction needs finite quotients
            const float most = 8.0f * d;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = fminf(fmaxf(v[e], -most), most);
          }
          codes = codes_of_quotient(v, d, __fdiv_rn(1.0f, d));
        }
      } else {
        // used is even, so both threads of a block are here
        amax = max_nan(amax, __shfl_xor_sync(3u << (lane & ~1), amax, 1));
        const uint32_t e = __float_as_uint(amax) >> 23;
        scale = e == 0xff ? 0xff : e > 2 ? e - 2 : 0;
        if (scale != 0xff) {
          const float up = __uint_as_float((254 - scale) << 23);  // 1 / scale
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = mul_exact(v[i], up);
          codes = make_uint2(to_e2m1x8(v), to_e2m1x8(v + 8));
        }
      }
      *reinterpret_cast<uint2*>(p.codes + row * (p.K / 2) + u * 8) = codes;
    }
    const int j = FORMAT == 0 ? lane & 3 : (lane >> 1) & 3;
    uint32_t word = scale << (8 * j);
#pragma unroll
    for (int o = FORMAT == 0 ? 1 : 2; o < kUnits; o <<= 1) word |= __shfl_xor_sync(peers, word, o);
    if ((lane & (kUnits - 1)) == 0)
      *reinterpret_cast<uint32_t*>(p.scales + scale_word(row, u / kUnits, p.tiles)) = word;
  }
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                                pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// The value of a code times two, a whole number: 0, 1, 2, 3, 4, 6, 8, 12.
__device__ __forceinline__ float twice_e2m1(uint32_t c) {
  const uint32_t m = c & 7, v = m < 4 ? m : (2 + (m & 1)) << (m >> 1) >> 1;
  return (c & 8) != 0 ? -(float)v : (float)v;
}

template <typename T, int FORMAT>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const float* __restrict__ tensor_scale, T* __restrict__ out, int rows, int K, int tiles, int width) {
  pdl_launch_dependents();
  pdl_wait();
  const float ts = FORMAT == 0 ? *tensor_scale : 1.0f;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / width) + threadIdx.x / width;
  if (row >= rows) return;
  for (int u = threadIdx.x % width; u < K / 16; u += width) {
    const uint2 c = *reinterpret_cast<const uint2*>(codes + row * (K / 2) + u * 8);
    const int block = FORMAT == 0 ? u : u >> 1;
    const uint32_t b = scales[scale_word(row, block >> 2, tiles) + (block & 3)];
    const float s = FORMAT == 0 ? of_e4m3(b) : of_e8m0(b);
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float q = twice_e2m1((e < 8 ? c.x : c.y) >> (4 * (e & 7)));
      // NVFP4: half of a code times an E4M3 is exact, the tensor's scale rounds once
      v[e] = FORMAT == 0 ? mul_exact(q * (0.5f * s), ts) : mul_exact(q * 0.5f, s);
    }
    store16(out + row * K + u * 16, v);
  }
}

int width_of(int units) {
  int w = 8;
  while (w < units && w < kThreads) w *= 2;
  return w;
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
  const int per = kThreads / p.width;
  const int64_t padded = ((int64_t)rows + 127) / 128 * 128;
  // (of no rows only the scale is written)
  const dim3 grid((unsigned)std::max<int64_t>(1, (padded + per - 1) / per)), block(kThreads);
  if (format == 0)
    return f32 ? launch_pdl(quantize_kernel<float, 0>, grid, block, 0, st, p)
               : launch_pdl(quantize_kernel<__nv_bfloat16, 0>, grid, block, 0, st, p);
  return f32 ? launch_pdl(quantize_kernel<float, 1>, grid, block, 0, st, p)
             : launch_pdl(quantize_kernel<__nv_bfloat16, 1>, grid, block, 0, st, p);
}

cudaError_t fp4_dequantize_launch(const void* codes, const void* scales, const float* tensor_scale, void* out, int rows,
                                  int K, int format, int dtype, cudaStream_t st) {
  const int tiles = k_tiles(K, format), width = width_of(K / 16), per = kThreads / width;
  const dim3 grid((unsigned)(((int64_t)rows + per - 1) / per)), block(kThreads);
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
