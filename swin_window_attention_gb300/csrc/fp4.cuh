// Microscaled 4-bit floating point: E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives),
// two to a byte, the even one in the low half, and a scale for each block of consecutive elements of
// a row:
// * NVFP4: blocks of 16 with an E4M3 scale, and one fp32 scale of the whole tensor;
// * MXFP4: blocks of 32 with a power of two (E8M0).
// The scales lie as the tensor core's scale memory wants them: tiles of 128 rows by 4 blocks,
// 512 bytes each, the scale of row r and block j of a tile at (r % 32) * 16 + (r / 32) * 4 + j, tiles of
// the same rows one behind the other. Rows and blocks past the end are zero.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace swin {

// One operand of a product: [rows, K] codes, their scales, and of NVFP4 the tensor's scale (device).
struct Fp4Operand {
  const void *codes, *scales;
  const float* tensor_scale;
};

namespace fp4 {

constexpr int kTileBytes = 512;

__host__ __device__ constexpr int block_of(int format) { return format == 0 ? 16 : 32; }
// Scale tiles along a row.
__host__ __device__ constexpr int k_tiles(int K, int format) { return (K / block_of(format) + 3) / 4; }
inline size_t scale_bytes(int64_t rows, int K, int format) {
  return (size_t)((rows + 127) / 128) * k_tiles(K, format) * kTileBytes;
}
// Where the four scales of the blocks 4 t .. 4 t + 3 of a row lie.
__device__ __forceinline__ int64_t scale_word(int64_t row, int t, int tiles) {
  const int r = (int)(row & 127);
  return ((row >> 7) * tiles + t) * kTileBytes + (r & 31) * 16 + (r >> 5) * 4;
}

}  // namespace fp4
}  // namespace swin
