// A dense layer on microscaled 4-bit operands: what its two forms (linear_fp4.cu: tiles;
// linear_fp4_few.cu: few tokens) share.
#pragma once

#include <cfloat>

#include "fp4.cuh"
#include "product.cuh"

namespace swin {

// The cluster-per-tile form for few tokens (linear_fp4_few.cu): TN tokens and 128 output channels per tile, `cluster` CTAs to
// a tile, each over its part of K, the largest cluster with which every tile is resident at once. `cost` estimates the
// time in SM clocks, on codes; chunk_rounds: the chunks that a CTA takes one after the other.
struct FewFp4Tiling {
  int TN, n_tiles, t_tiles, chunks, cluster;
  double chunk_rounds, cost;
};
FewFp4Tiling few_fp4_tiling(int64_t T, int N, int K);
// x: codes (x_bytes 1, with their scales), or bf16 or fp32 values (2, 4), which are quantised on the way; x_scale: the
// tensor's scale of NVFP4.
cudaError_t linear_fp4_few_launch(const FewFp4Tiling& t, const void* x, const void* x_scales, int x_bytes, const float* x_scale,
                                  const Fp4Operand& w, const float* b, const void* residual, void* y, int T, int K, int N,
                                  int format, int act, int* status, cudaStream_t st);

namespace fp4 {

// A chunk of K is 256 elements, a 128-byte row of codes, and takes four MMAs of 64; their scales are four
// tiles of NVFP4 (a tile a MMA) or two of MXFP4 (a tile for two).
constexpr int kChunk = 256, kStep = 64;
__host__ __device__ constexpr int chunk_tiles(int format) { return format == 0 ? 4 : 2; }

// Instruction descriptor of the block-scaled 4-bit kinds: A and B E2M1 (format 1 at bits 7 and 10), N >> 3 from
// bit 17, scale type at bit 23 (0 E4M3, 1 E8M0), M >> 4 from bit 24; bits 4 and 29 select the scales of
// B and A within their 32-bit words (MXFP4: 0 or 2 for the two MMAs of a tile).
__host__ __device__ constexpr uint32_t idesc(int m, int n, int format) {
  return 1u << 7 | 1u << 10 | (uint32_t)(n >> 3) << 17 | (format == 0 ? 0u : 1u << 23) | (uint32_t)(m >> 4) << 24;
}
__host__ __device__ constexpr uint32_t idesc_second_half() { return 2u << 4 | 2u << 29; }

#ifdef __CUDACC__
// D[tmem] (+)= (A sA)(B sB)^T on 4-bit operands, K = 64; sa and sb are the scales' columns.
template <int CG, int FORMAT>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t sa, uint32_t sb,
                                    bool accumulate) {
#define SWIN_FP4_MMA(GROUP, KIND)                                                                                    \
  asm volatile(                                                                                                      \
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.u32 p, %7, 0;\n mov.b64 da, {%1, %3};\n mov.b64 db, {%2, %3};\n" \
      " tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], da, db, %4, [%5], [%6], p;\n}\n" ::"r"(d),             \
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate ? 1u : 0u)                                \
      : "memory")
  if constexpr (CG == 1 && FORMAT == 0) SWIN_FP4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (CG == 2 && FORMAT == 0) SWIN_FP4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (CG == 1 && FORMAT == 1) SWIN_FP4_MMA("1", "mxf4.block_scale.scale_vec::2X");
  if constexpr (CG == 2 && FORMAT == 1) SWIN_FP4_MMA("2", "mxf4.block_scale.scale_vec::2X");
#undef SWIN_FP4_MMA
}
// A scale tile (32 rows of 16 bytes, each the four words of rows r, r + 32, r + 64, r + 96) from shared memory
// to four columns of tensor memory, the same in each quadrant of lanes (of both CTAs of a pair).
// `lo` is the low word of the tile's descriptor.
constexpr uint32_t kScaleHi = 128 >> 4 | 1u << 14;  // groups of eight rows 128 bytes apart, no swizzle
__device__ __forceinline__ uint32_t scale_lo(uint32_t smem) { return ((smem >> 4) & 0x3FFFu) | 1u << 16; }
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t lo) {
  if constexpr (CG == 2)
    asm volatile("{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n}\n" ::"r"(taddr),
                 "r"(lo), "r"(kScaleHi)
                 : "memory");
  else
    asm volatile("{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n}\n" ::"r"(taddr),
                 "r"(lo), "r"(kScaleHi)
                 : "memory");
}
// The two tensors' scales as two factors of a sum: x the first, y the rest. The first is 1 unless fp32 does not hold their
// product; then it is a power of two, by which a sum (2^-20 to 2^38 in size, or zero) is multiplied exactly, and the rest is
// held. (A product of scales above 2^192 makes each sum but zero infinite, as the largest number in its place does.)
__device__ __forceinline__ float2 tensor_scales(float sx, float sw) {
  const float both = sx * sw, up = both > 1.0f ? 0x1p32f : 0x1p-32f, down = both > 1.0f ? 0x1p-32f : 0x1p32f;
  const bool held = !(both < FLT_MIN || both > FLT_MAX);  // (NaN as it is)
  return make_float2(held ? 1.0f : up * up, held ? both : fminf((sx * down) * (sw * down), FLT_MAX));
}
#endif

namespace {

// Tensor map of an operand's codes, in 128-byte rows.
inline cudaError_t encode_codes(CUtensorMap* codes, const Fp4Operand& x, int64_t rows, int K, int box_rows) {
  const prod::Matrix m{x.codes, rows, K / 2, K / 2, 0};
  return prod::encode_3d(codes, m, 1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, box_rows, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

}  // namespace
}  // namespace fp4
}  // namespace swin
