// Quantisation of sixteen consecutive elements by a thread, shared by the kernels that write 4-bit operands to memory
// (fp4.cu) and the one that makes them where they are multiplied (linear_fp4_few.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"

namespace swin {
namespace fp4 {

// Products and their sums that keep subnormals (the library is built to flush them).
__device__ __forceinline__ float mul_exact(float a, float b) {
  float r;
  asm("mul.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float fma_exact(float a, float b, float c) {
  float r;
  asm("fma.rn.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma2_exact(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// Eight values to eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t to_e2m1x8(const float2* v) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}
// Eight codes to eight halves (exact).
__device__ __forceinline__ void of_e2m1x8(uint32_t c, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
}
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xff;
}
// An E4M3 without a sign, 0x7f is NaN.
__device__ __forceinline__ float of_e4m3(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)b));
  return __half2float(__ushort_as_half((uint16_t)h));
}
// 2^(b - 127); 0xff is NaN.
__device__ __forceinline__ float of_e8m0(uint32_t b) {
  return __uint_as_float(b == 0xff ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
}

// 16 elements as they lie in memory.
template <typename T>
struct Raw16 {
  uint4 w[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw16<T> load16(const T* p) {
  Raw16<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void unpack16(const Raw16<__nv_bfloat16>& r, float2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t in[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * i + k] = make_float2(__uint_as_float(in[k] << 16), __uint_as_float(in[k] & 0xffff0000u));
  }
}
__device__ __forceinline__ void unpack16(const Raw16<float>& r, float2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = make_float2(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
    v[2 * i + 1] = make_float2(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
  }
}
// Their largest magnitude; above infinity's bits where there is a NaN. Magnitudes order as their bits do.
__device__ __forceinline__ uint32_t amax_bits(const Raw16<__nv_bfloat16>& r) {
  constexpr uint32_t k = 0x7fff7fffu;
  uint32_t m = __vimax3_u16x2(r.w[0].x & k, r.w[0].y & k, r.w[0].z & k);
  m = __vimax3_u16x2(m, r.w[0].w & k, r.w[1].x & k);
  m = __vimax3_u16x2(m, r.w[1].y & k, r.w[1].z & k);
  m = __vimax3_u16x2(m, m, r.w[1].w & k);
  return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ uint32_t amax_bits(const Raw16<float>& r) {
  constexpr uint32_t k = 0x7fffffffu;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = __vimax3_u32(m, r.w[i].x & k, r.w[i].y & k);
    m = __vimax3_u32(m, r.w[i].z & k, r.w[i].w & k);
  }
  return m;
}
constexpr uint32_t kInfinity = 0x7f800000u;

// 1 / d to nearest, but for a unit in the last place in rare cases: the hardware's reciprocal, corrected once.
__device__ __forceinline__ float reciprocal(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(d));
  return fmaf(fmaf(-d, r, 1.0f), r, r);
}
// x / d, rounded to nearest: the product with the reciprocal r, corrected by its remainder, which an fma gives exactly
// (Markstein, 1990). An exact quotient comes out exact, so ties between codes are met as a division would. The remainder
// is some 2^-24 of x: below a scale of the tensor of 2^-97 it is subnormal, and kept.
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q = x * r;
  return fma_exact(fma_exact(-q, d, x), r, q);
}
// Codes of the 16 values x of an NVFP4 block, the quotients by d.
__device__ __forceinline__ uint2 codes_of_quotient(const float2 (&x)[8], float d, float r) {
  float2 q[8];
  const float2 r2 = make_float2(r, r), d2 = make_float2(-d, -d);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 q0 = __fmul2_rn(x[e], r2);
    q[e] = fma2_exact(fma2_exact(q0, d2, x[e]), r2, q0);
  }
  return make_uint2(to_e2m1x8(q), to_e2m1x8(q + 4));
}

constexpr float kSixth = 0.16666667163372039794921875f;  // 1 / 6, to nearest

// Codes and scale (E4M3 or E8M0) of 16 elements; of MXFP4 two neighbouring threads share a block, and `pair` names the
// lanes of both. r_ts: 1 / ts.
template <int FORMAT, typename T>
__device__ __forceinline__ uint2 quantize16(const Raw16<T>& raw, float ts, float r_ts, unsigned pair, uint32_t& scale) {
  uint32_t bits = amax_bits(raw);
  float2 v[8];
  unpack16(raw, v);
  uint2 codes = make_uint2(0, 0);
  if constexpr (FORMAT == 0) {
    // a given scale may be too small by any factor: the corrections need finite quotients, and from 448 on the scale is the
    // largest, so the ratio is formed of 512 ts at most (an infinite one would be corrected to NaN), and the values are cut
    // to 8 d, whose codes are the largest
    const float sixth = fminf(quotient(__uint_as_float(bits), 6.0f, kSixth), 512.0f * ts);
    const float ratio = quotient(sixth, ts, r_ts);
    scale = bits < kInfinity ? to_e4m3(ratio) : 0x7f;
    const float s = of_e4m3(scale), d = s * ts;
    if (s > 0.0f) {
      if (ratio > 448.0f) {
        const float most = 8.0f * d;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = make_float2(fminf(fmaxf(v[e].x, -most), most), fminf(fmaxf(v[e].y, -most), most));
      }
      codes = codes_of_quotient(v, d, reciprocal(d));
    }
  } else {
    bits = max(bits, __shfl_xor_sync(pair, bits, 1));
    const uint32_t e = bits >> 23;
    scale = e == 0xff ? 0xff : e > 2 ? e - 2 : 0;
    if (scale != 0xff) {
      const float up = __uint_as_float((254 - scale) << 23);  // 1 / scale
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = make_float2(mul_exact(v[i].x, up), mul_exact(v[i].y, up));
      codes = make_uint2(to_e2m1x8(v), to_e2m1x8(v + 4));
    }
  }
  return codes;
}

}  // namespace fp4
}  // namespace swin
