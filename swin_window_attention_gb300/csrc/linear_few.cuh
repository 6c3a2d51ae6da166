// The cluster-per-tile form of linear and linear_bwd_data (linear_few.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace swin {

// TN tokens and 128 output channels per tile, `cluster` CTAs to a tile, each over its part of K:
// the largest cluster with which every tile is resident at once, of two chunks per CTA at least
// (one more CTA per tile than fits costs a second round: 48 tiles of 24 chunks took 12.6 us in
// clusters of three, 7.3 us in pairs). `cost` estimates the time in SM clocks, as measured: 7000
// for the launch and the pipeline's ends, the chunks' loads, 500 per CTA of the cluster and 40
// per token for the sum over it.
struct FewTiling {
  int TN, n_tiles, t_tiles, chunks, cluster;
  double cost;
};
FewTiling few_tiling(int64_t T, int N, int64_t K);

cudaError_t linear_few_launch(const FewTiling& t, const void* x, const void* w, const float* b, const void* residual,
                              void* y, void* pre, int T, int K, int N, int act, int* status, cudaStream_t st);
cudaError_t linear_bwd_data_few_launch(const FewTiling& t, const void* dy, const void* w, const void* pre, void* dx,
                                       int T, int K, int N, int act, int* status, cudaStream_t st);

}  // namespace swin
