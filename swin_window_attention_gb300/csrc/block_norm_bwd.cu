// The gradients of block_norm: the parameter gradients from the blocks' sums, and the entry (block_norm_bwd.cuh has the
// formulas and the kernel over the rows).
#include "block_norm_bwd.cuh"

namespace swin {

cudaError_t block_norm_bwd_bf16(const NormBwdParams& p, cudaStream_t st);
cudaError_t block_norm_bwd_fp32(const NormBwdParams& p, cudaStream_t st);

namespace {

struct ParamGrads {
  const float *post_w, *post_b, *gate;
  float *pre_w_out, *pre_b_out, *post_w_out, *post_b_out, *gate_out;
  bool has_post, accumulate;
};

// The parameter gradients of eight channels: the blocks' sums, 64 threads a channel each over every 64th block, then
// in order. (32 channels and 16 threads each left most SMs idle: of 760 blocks' sums of 768 channels 30 us.)
constexpr int kSumCols = 8, kSumRows = 64;
__global__ void __launch_bounds__(kSumCols * kSumRows)
    param_grads_kernel(const float* __restrict__ partial, int blocks, int C, const ParamGrads g) {
  __shared__ float part[kSums][kSumRows][kSumCols];
  pdl_launch_dependents();
  pdl_wait();
  const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols, c = blockIdx.x * kSumCols + x;
  float s[kSums] = {};
#pragma unroll 4
  for (int b = y; b < blocks; b += kSumRows) {
#pragma unroll
    for (int k = 0; k < kSums; ++k) s[k] += __ldcg(partial + ((int64_t)b * kSums + k) * C + c);
  }
#pragma unroll
  for (int k = 0; k < kSums; ++k) part[k][y][x] = s[k];
  __syncthreads();
  if (y >= kSums) return;
  // one thread a sum and channel, then one a channel
  float a = 0.0f;
#pragma unroll 16
  for (int i = 0; i < kSumRows; ++i) a += part[y][i][x];
  __syncwarp();
  part[y][0][x] = a;
  __syncwarp();
  if (y != 0) return;
#pragma unroll
  for (int k = 0; k < kSums; ++k) s[k] = part[k][0][x];
  auto put = [&](float* out, float v) {
    if (out != nullptr) out[c] = g.accumulate ? out[c] + v : v;
  };
  put(g.pre_w_out, s[0]);
  put(g.pre_b_out, s[1]);
  const float gate = g.gate != nullptr ? g.gate[c] : 1.0f;
  put(g.post_w_out, gate * s[2]);
  put(g.post_b_out, gate * s[3]);
  put(g.gate_out, g.has_post ? fmaf(g.post_w[c], s[2], (g.post_b != nullptr ? g.post_b[c] : 0.0f) * s[3]) : s[2]);
}

}  // namespace

size_t block_norm_bwd_workspace_bytes(int tokens, int C) {
  const int blocks = std::max(blocks_of(tokens, shape_of(C, false)), blocks_of(tokens, shape_of(C, true)));
  return std::max<size_t>(256, (size_t)blocks * kSums * C * 4);
}

cudaError_t block_norm_bwd_launch(const void* y, const void* f, const void* dh, const void* dy, const float* pre_w,
                                  const float* post_w, const float* post_b, const float* gate, const float* keep,
                                  void* dx, void* df, float* dpre_w, float* dpre_b, float* dpost_w, float* dpost_b,
                                  float* dgate, int tokens, int C, int samples, int dtype, int kind, float alpha,
                                  float eps, int accumulate, void* workspace, cudaStream_t st) {
  const Shape s = shape_of(C, post_w != nullptr);
  const int blocks = blocks_of(tokens, s);
  BwdParams p{};
  p.y = y;
  p.dy = dy;
  p.f = static_cast<const __nv_bfloat16*>(f);
  p.dh = static_cast<const __nv_bfloat16*>(dh);
  p.pre_w = pre_w;
  p.post_w = post_w;
  p.gate = gate;
  p.keep = keep;
  p.dx = dx;
  p.df = static_cast<__nv_bfloat16*>(df);
  p.partial = static_cast<float*>(workspace);
  p.rows = tokens;
  p.C = C;
  p.per_sample = keep != nullptr && tokens > 0 ? tokens / samples : 1;
  p.rms = kind == SWIN_WATTN_NORM_RMS;
  p.alpha = f != nullptr ? alpha : 1.0f;  // (without f the forward does not use it)
  p.eps = eps;
  p.inv_c = 1.0f / (float)C;
  if (tokens > 0) {
    const cudaError_t e = dtype == SWIN_WATTN_FP32 ? block_norm_bwd_fp32(p, st) : block_norm_bwd_bf16(p, st);
    if (e != cudaSuccess) return e;
  }
  ParamGrads g{post_w, post_b, gate, dpre_w, dpre_b, dpost_w, dpost_b, dgate, post_w != nullptr, accumulate != 0};
  if (dpre_w == nullptr && dpre_b == nullptr && dpost_w == nullptr && dpost_b == nullptr && dgate == nullptr)
    return cudaSuccess;
  return launch_pdl(param_grads_kernel, dim3(C / kSumCols), dim3(kSumCols * kSumRows), 0, st, (const float*)p.partial, blocks, C, g);
}

}  // namespace swin
