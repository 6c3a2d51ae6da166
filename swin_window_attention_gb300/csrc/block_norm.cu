// The residual sum around a block with its gate and the norms on both sides:
//   u = post(f) or f,   y = alpha x + keep[sample] gate[channel] u,   h = pre(y)
// pre is the norm before the next block, post the one after this block (a res-post-norm block
// has both); either may be absent, and without f the kernel is a plain norm of x.
// One pass: a row is read once, both norms' sums are taken in registers, y and h are written.
// h is normalised from y in fp32, before y is rounded for its store: its one rounding is the one
// to bf16.
#include "block_norm.cuh"

namespace swin {

namespace {

using namespace norm;

struct FwdParams {
  const void* x;
  const __nv_bfloat16* f;
  const float *pre_w, *pre_b, *post_w, *post_b, *gate, *keep;
  void* y;
  __nv_bfloat16* h;
  int rows, C, per_sample;
  bool rms;
  float alpha, eps, inv_c;
};

template <typename S, int LANES, int CH>
__global__ void __launch_bounds__(LANES == 0 ? 512 : kThreads) block_norm_kernel(const FwdParams p) {
  __shared__ float2 slots[LANES == 0 ? 32 : 1];
  pdl_launch_dependents();
  pdl_wait();
  RowSum<LANES> sum{slots};
  const int width = LANES == 0 ? blockDim.x : LANES;
  const int lane = LANES == 0 ? threadIdx.x : threadIdx.x % width;
  const int64_t own = (int64_t)blockIdx.x * (blockDim.x / width) + threadIdx.x / width;
  const bool valid = own < p.rows;
  const int64_t row = valid ? own : p.rows - 1;  // every thread takes part in the sums
  int col[CH];
  bool in[CH];
  float v[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    col[j] = (j * width + lane) * 8;
    in[j] = col[j] < p.C;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
    if (in[j]) load8(static_cast<const S*>(p.x) + row * p.C + col[j], v[j]);
  }
  if (p.f != nullptr) {
    float u[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[j][e] = 0.0f;
      if (in[j]) load8(p.f + row * p.C + col[j], u[j]);
    }
    const float keep = p.keep != nullptr ? p.keep[(unsigned)row / (unsigned)p.per_sample] : 1.0f;
    if (p.post_w != nullptr) normalise<LANES, CH>(u, in, p.rms, p.inv_c, p.eps, sum);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if (!in[j]) continue;
      float a[8];
      if (p.post_w != nullptr) {
        load_param8(p.post_w + col[j], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[j][e] *= a[e];
        if (p.post_b != nullptr) {
          load_param8(p.post_b + col[j], a);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[j][e] += a[e];
        }
      }
      if (p.gate != nullptr) {
        load_param8(p.gate + col[j], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[j][e] *= a[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = fmaf(p.alpha, v[j][e], keep * u[j][e]);
      if (valid) store8(static_cast<S*>(p.y) + row * p.C + col[j], v[j]);
    }
  }
  if (p.pre_w == nullptr) return;
  normalise<LANES, CH>(v, in, p.rms, p.inv_c, p.eps, sum);
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    if (!in[j]) continue;
    float a[8];
    load_param8(p.pre_w + col[j], a);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] *= a[e];
    if (p.pre_b != nullptr) {
      load_param8(p.pre_b + col[j], a);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] += a[e];
    }
    if (valid) store8(p.h + row * p.C + col[j], v[j]);
  }
}

template <typename S>
cudaError_t launch(const FwdParams& p, cudaStream_t st) {
  const Shape s = shape_of(p.C);
  const dim3 grid((unsigned)(((int64_t)p.rows + s.rows_per_block - 1) / s.rows_per_block)), block(s.threads);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, block, 0, st, p); };
  switch (s.lanes * 4 + s.chunks) {
    case 4 * 4 + 2: return go(block_norm_kernel<S, 4, 2>);
    case 4 * 4 + 3: return go(block_norm_kernel<S, 4, 3>);
    case 8 * 4 + 2: return go(block_norm_kernel<S, 8, 2>);
    case 8 * 4 + 3: return go(block_norm_kernel<S, 8, 3>);
    case 16 * 4 + 2: return go(block_norm_kernel<S, 16, 2>);
    case 16 * 4 + 3: return go(block_norm_kernel<S, 16, 3>);
    case 32 * 4 + 2: return go(block_norm_kernel<S, 32, 2>);
    case 32 * 4 + 3: return go(block_norm_kernel<S, 32, 3>);
    default: return go(block_norm_kernel<S, 0, 2>);
  }
}

}  // namespace

cudaError_t block_norm_launch(const void* x, const void* f, const float* pre_w, const float* pre_b, const float* post_w,
                              const float* post_b, const float* gate, const float* keep, void* y, void* h, int tokens,
                              int C, int samples, int dtype, int kind, float alpha, float eps, cudaStream_t st) {
  FwdParams p{};
  p.x = x;
  p.f = static_cast<const __nv_bfloat16*>(f);
  p.pre_w = pre_w;
  p.pre_b = pre_b;
  p.post_w = post_w;
  p.post_b = post_b;
  p.gate = gate;
  p.keep = keep;
  p.y = y;
  p.h = static_cast<__nv_bfloat16*>(h);
  p.rows = tokens;
  p.C = C;
  p.per_sample = keep != nullptr ? tokens / samples : 1;
  p.rms = kind == SWIN_WATTN_NORM_RMS;
  p.alpha = alpha;
  p.eps = eps;
  p.inv_c = 1.0f / (float)C;
  return dtype == SWIN_WATTN_FP32 ? launch<float>(p, st) : launch<__nv_bfloat16>(p, st);
}

}  // namespace swin
