// What the two forms of the Newton-Schulz update share: the coefficients, the scale of the
// matrices held in fp16, the norm and the reads of G.
#pragma once

#include "product.cuh"

namespace swin {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
// Of the fp16 matrices held: A and B, and X, which is held in two parts, its rounding to fp16 and
// what that leaves: together 22 bits, down to 2^-39.
// (In one part X came out percents off where G is of low rank or its singular values fall off: the
// rounding's noise lies in every direction, and in those that G does not have, the steps multiply it
// by 3.44 each, 483 in five. Rank 49 of 512 x 2048: 2.4e-2 of the exact result; in two parts 1.2e-3.
// A and B act on X from one side, so the noise of their roundings stays within the directions of X.)
constexpr float kScale = 256.0f, kScaleX = 16384.0f;

// Of a step's roundings to fp16 those of the diagonals of A and of B = a I + b A + c A^2 cost most:
// an entry of B's multiplies a whole row of X. So
// * A' = A - mu I is held instead of A, with mu near the middle of A's diagonal:
//     B = e I + (b + 2 c mu) A' + c A'^2,   e = a + b mu + c mu^2;
// * where B's diagonal entry was rounded, the row of X it belongs to (of B X; the column of X B) is
//   multiplied by the quotient of the exact entry and the rounded one, in fp32 with the product's
//   own scaling. That is exact where B is diagonal, and near it while the singular values
//   rise, when nothing later takes the error back.
// (The error of the result over that of rounding the exact one to bf16, on spectra from flat to
// 1 / sqrt(k), three to twelve steps: 1.13 to 2.1 without either, 1.07 to 1.4 with both.)
struct NsStep {
  float mu, b, e;
};
__host__ __device__ __forceinline__ NsStep ns_step(float mu) {
  return {mu, kNsB + 2.0f * kNsC * mu, kNsA + mu * (kNsB + mu * kNsC)};
}
// The shifts follow the squares of the singular values as the steps take them up: were they all
// equal, A's diagonal would begin at 1 / m; with a few larger ones, as gradients have, most are
// below that (0.36). From 0.12 on, a step takes them to the final band, whose middle is near 0.75.
__host__ __device__ __forceinline__ float first_shift(int m) { return 0.36f / m; }
__host__ __device__ __forceinline__ float next_shift(float mu) {
  const float p = kNsA + mu * (kNsB + mu * kNsC);
  return mu > 0.12f ? 0.75f : mu * p * p;
}

// The two parts of two values of X.
__device__ __forceinline__ void two_parts(float2 v, uint32_t& high, uint32_t& low) {
  high = prod::pack_f16(v.x, v.y);
  const float2 rest = fsub2(v, prod::unpack_f16(high));
  low = prod::pack_f16(rest.x, rest.y);
}

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

// A plain fp32 sum of squares is the norm's if it comes out between these: then no square has
// overflowed, and those below the smallest fp32 (2^28 of them at most) are nothing beside it. NaN
// and infinities are outside too.
__device__ __forceinline__ bool plain_sum_holds(float s) { return s >= 0x1p-60f && s <= 0x1p96f; }

// Else squares are summed apart for values in [2^-48, 2^48), for larger ones times 2^-64 (NaN
// and infinity too) and for smaller ones times 2^64, so that no square overflows or is lost
// where the norm is a normal number. (Subnormal values count as zero. Summing every matrix
// this way took 2.5 us of 27 for one 96 x 384.)
struct Squares {
  float mid, big, small;
};
constexpr float kTwo64 = 0x1p64f;
__device__ __forceinline__ void add_square(float v, Squares& s) {
  const float a = fabsf(v);
  if (a < 0x1p-48f) {
    const float x = v * kTwo64;
    s.small = fmaf(x, x, s.small);
  } else if (a < 0x1p48f) {
    s.mid = fmaf(v, v, s.mid);
  } else {
    const float x = v * (1.0f / kTwo64);
    s.big = fmaf(x, x, s.big);
  }
}
// Eight squares to a plain sum's two halves.
__device__ __forceinline__ void add_plain(const float (&v)[8], float2& s) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) s = __ffma2_rn(make_float2(v[e], v[e + 1]), make_float2(v[e], v[e + 1]), s);
}
__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
__device__ __forceinline__ void add(Squares& s, const Squares& o) {
  s.mid += o.mid;
  s.big += o.big;
  s.small += o.small;
}
__device__ __forceinline__ Squares warp_sum(const Squares& s) { return {warp_sum(s.mid), warp_sum(s.big), warp_sum(s.small)}; }
// The norm: each sum joins the next larger one in that one's scale (what of it is lost
// there is below that sum's rounding).
__device__ __forceinline__ float norm_of(const Squares& s) {
  constexpr float k = 1.0f / kTwo64;
  if (s.big != 0.0f) return sqrtf(s.big + s.mid * k * k) * kTwo64;
  if (s.mid != 0.0f) return sqrtf(s.mid + s.small * k * k);
  return sqrtf(s.small) * k;
}
// X = kScaleX G / (|G| + eps) is G * pre * inv: 1 / (|G| + eps) itself can overflow.
struct Inverse {
  float pre, inv;
};
__device__ __forceinline__ Inverse inverse_of(const Squares& s, float eps) {
  const float d = norm_of(s) + eps, pre = d < 1.0f / kTwo64 ? kTwo64 : 1.0f;
  return {pre, __fdiv_rn(kScaleX, d * pre)};
}

}  // namespace swin
