// A dense layer on microscaled 4-bit operands: what its two forms (linear_fp4.cu: tiles;
// linear_fp4_few.cu: few tokens) share.
#pragma once

#include "fp4.cuh"
#include "product.cuh"

namespace swin {

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
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t smem) {
  const uint64_t desc = tc::sdesc(smem, 16, 128);
  if constexpr (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}
#endif

namespace {

// Tensor maps of an operand: 128-byte rows of codes, and its scale tiles.
inline cudaError_t encode_operand(CUtensorMap* codes, CUtensorMap* scales, const Fp4Operand& x, int64_t rows, int K,
                                  int format, int box_rows) {
  const prod::Matrix m{x.codes, rows, K / 2, K / 2, 0};
  const int tiles = k_tiles(K, format);
  const prod::Matrix s{x.scales, tiles, kTileBytes / 4, kTileBytes / 4, (int64_t)tiles * (kTileBytes / 4)};
  const cudaError_t e = prod::encode_3d(codes, m, 1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, box_rows,
                                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (e != cudaSuccess) return e;
  return prod::encode_3d(scales, s, (int)((rows + 127) / 128), CU_TENSOR_MAP_DATA_TYPE_INT32, 4, kTileBytes / 4,
                         chunk_tiles(format), CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

}  // namespace
}  // namespace fp4
}  // namespace swin
