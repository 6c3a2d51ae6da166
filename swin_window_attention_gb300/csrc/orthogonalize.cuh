// What the two forms of the Newton-Schulz update share: the coefficients, the scale of the
// matrices held in fp16, the norm and the reads of G.
#pragma once

#include "product.cuh"

namespace swin {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr float kScale = 256.0f;  // of every fp16 matrix held

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
// Eight consecutive values, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = prod::unpack_bf16(in[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Squares are summed apart for values below 2^48 (lo) and, times 2^-64, for the others (hi:
// NaN and infinity too), so that neither sum overflows where the norm does not.
__device__ __forceinline__ void add_square(float v, float& lo, float& hi) {
  if (fabsf(v) < 281474976710656.0f) {
    lo = fmaf(v, v, lo);
  } else {
    const float s = v * 5.421010862427522e-20f;
    hi = fmaf(s, s, hi);
  }
}
// The norm of both sums; where the second is not empty the first is added in its scale.
__device__ __forceinline__ float norm_of(float lo, float hi) {
  return hi == 0.0f ? sqrtf(lo)
                    : sqrtf(hi + lo * 5.421010862427522e-20f * 5.421010862427522e-20f) * 18446744073709551616.0f;
}

}  // namespace swin
