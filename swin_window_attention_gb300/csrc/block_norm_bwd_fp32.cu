// The gradients of block_norm for a residual stream in fp32 (block_norm_bwd.cuh).
#include "block_norm_bwd.cuh"

namespace swin {

cudaError_t block_norm_bwd_fp32(const NormBwdParams& p, cudaStream_t st) {
  const Shape s = shape_of(p.C, p.post_w != nullptr);
  return launch<float>(p, s, blocks_of(p.rows, s), st);
}

}  // namespace swin
