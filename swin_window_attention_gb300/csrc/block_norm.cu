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
  bool rms, vec;
  float alpha, eps, inv_c;
};

// A group takes kRows rows at a time: the parameters, as many bytes of a row as its own in bf16, are read from the
// caches once for both, and one round of sums serves both. (A row at a time, 100352 x 192 with both norms, gate
// and depth took 38 us, the load and store units 72 % busy; 25088 x 768 with gate 32.6 us instead of 30.3.) One row where a
// thread has three or four chunks, whose registers for two leave one block on an SM (2400 x 8192: 51 us, 38 with one).
__host__ __device__ constexpr int rows_of(int lanes, int chunks) { return lanes == 0 && chunks >= 3 ? 1 : 2; }

constexpr int kThreads = 256;  // of a block of groups that lie in warps

// Of the least capacity: two or three chunks in a warp; in a block two up to 4096 channels, three or four above. (Four in
// a warp: 37632 x 512 53 us, two in a block 36.)
Shape shape_of(int C) {
  const int n = C / kV;
  for (int lanes = 4; lanes <= 32; lanes *= 2)
    for (int ch = 2; ch <= 3; ++ch)
      if (n <= lanes * ch) return {lanes, ch, kThreads, kThreads / lanes};
  const auto threads = [&](int ch) { return ((n + ch - 1) / ch + 31) / 32 * 32; };
  int ch = 2;
  while (threads(ch) > 32 * kMaxWarps) ++ch;
  return {0, ch, threads(ch), 1};
}

template <typename S, int LANES, int CH>
__global__ void __launch_bounds__(LANES == 0 ? 32 * kMaxWarps : kThreads) block_norm_kernel(const FwdParams p) {
  __shared__ float2 slots[LANES == 0 ? 2 * kMaxWarps : 1];
  pdl_launch_dependents();
  pdl_wait();
  RowSum<LANES> sum{slots};
  const int width = LANES == 0 ? blockDim.x : LANES;
  const int lane = LANES == 0 ? threadIdx.x : threadIdx.x % width;
  const int groups = LANES == 0 ? 1 : kThreads / width;
  constexpr int kRows = rows_of(LANES, CH);
  int64_t row[kRows];  // neighbouring groups' first rows, then their second rows
  bool valid[kRows];
  int col[CH];
  bool in[CH];
  Four v[kRows][CH], u[kRows][CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    col[j] = (j * width + lane) * kV;
    in[j] = col[j] < p.C;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    row[k] = ((int64_t)blockIdx.x * kRows + k) * groups + (LANES == 0 ? 0 : threadIdx.x / width);
    valid[k] = row[k] < p.rows;
    const int64_t at = (valid[k] ? row[k] : p.rows - 1) * p.C;  // every thread takes part in the sums
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      v[k][j] = in[j] ? load4(static_cast<const S*>(p.x) + at + col[j]) : zeros();
      u[k][j] = in[j] && p.f != nullptr ? load4(p.f + at + col[j]) : zeros();
    }
  }
  if (p.f != nullptr) {
    float keep[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      keep[k] = p.keep != nullptr && valid[k] ? p.keep[(unsigned)row[k] / (unsigned)p.per_sample] : 1.0f;
    if (p.post_w != nullptr) {
      if constexpr (kRows == 2)
        normalise_both<LANES, CH>(u[0], u[1], in, p.rms, p.inv_c, p.eps, sum);
      else
        normalise<LANES, CH>(u[0], in, p.rms, p.inv_c, p.eps, sum);
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if (!in[j]) continue;
      if (p.post_w != nullptr) {
        const Four w = load_param4(p.post_w + col[j], p.vec);
        const Four b = p.post_b != nullptr ? load_param4(p.post_b + col[j], p.vec) : zeros();
#pragma unroll
        for (int k = 0; k < kRows; ++k) u[k][j] = fma(u[k][j], w, b);
      }
      if (p.gate != nullptr) {
        const Four w = load_param4(p.gate + col[j], p.vec);
#pragma unroll
        for (int k = 0; k < kRows; ++k) u[k][j] = mul(u[k][j], w);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        v[k][j] = fma(v[k][j], p.alpha, mul(u[k][j], keep[k]));
        if (valid[k]) store4(static_cast<S*>(p.y) + row[k] * p.C + col[j], v[k][j]);
      }
    }
  }
  if (p.pre_w == nullptr) return;
  if constexpr (kRows == 2)
    normalise_both<LANES, CH>(v[0], v[1], in, p.rms, p.inv_c, p.eps, sum);
  else
    normalise<LANES, CH>(v[0], in, p.rms, p.inv_c, p.eps, sum);
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    if (!in[j]) continue;
    const Four w = load_param4(p.pre_w + col[j], p.vec);
    const Four b = p.pre_b != nullptr ? load_param4(p.pre_b + col[j], p.vec) : zeros();
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (valid[k]) store4(p.h + row[k] * p.C + col[j], fma(v[k][j], w, b));
  }
}

template <typename S>
cudaError_t launch(const FwdParams& p, cudaStream_t st) {
  const Shape s = shape_of(p.C);
  const int per_block = s.rows_per_block * rows_of(s.lanes, s.chunks);
  const dim3 grid((unsigned)(((int64_t)p.rows + per_block - 1) / per_block)), block(s.threads);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, block, 0, st, p); };
  switch (s.lanes * 8 + s.chunks) {
    case 4 * 8 + 2: return go(block_norm_kernel<S, 4, 2>);
    case 4 * 8 + 3: return go(block_norm_kernel<S, 4, 3>);
    case 8 * 8 + 2: return go(block_norm_kernel<S, 8, 2>);
    case 8 * 8 + 3: return go(block_norm_kernel<S, 8, 3>);
    case 16 * 8 + 2: return go(block_norm_kernel<S, 16, 2>);
    case 16 * 8 + 3: return go(block_norm_kernel<S, 16, 3>);
    case 32 * 8 + 2: return go(block_norm_kernel<S, 32, 2>);
    case 32 * 8 + 3: return go(block_norm_kernel<S, 32, 3>);
    case 0 * 8 + 2: return go(block_norm_kernel<S, 0, 2>);
    case 0 * 8 + 3: return go(block_norm_kernel<S, 0, 3>);
    default: return go(block_norm_kernel<S, 0, 4>);
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
  p.vec = aligned16({pre_w, pre_b, post_w, post_b, gate});
  p.rms = kind == SWIN_WATTN_NORM_RMS;
  p.alpha = alpha;
  p.eps = eps;
  p.inv_c = 1.0f / (float)C;
  return dtype == SWIN_WATTN_FP32 ? launch<float>(p, st) : launch<__nv_bfloat16>(p, st);
}

}  // namespace swin
