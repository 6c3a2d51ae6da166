// Gradients of the residual sum around a block with its gate and norms (block_norm.cu). With
// yhat and fhat the normalised rows of y and f, recomputed from them, and r their factors:
//   g = dh pre_w,   dyt = dy + r_y (g - mean g - yhat mean(g yhat))      (RMS: without mean g)
//   dx = alpha dyt,   t = keep gate dyt post_w,   df = r_f (t - mean t - fhat mean(t fhat))
// and, as sums over the tokens,
//   dpre_w = sum dh yhat,  dpre_b = sum dh,  P = sum keep dyt fhat,  Q = sum keep dyt,
//   dpost_w = gate P,  dpost_b = gate Q,  dgate = post_w P + post_b Q   (without post: sum keep dyt f):
// four sums a channel give all five parameter gradients.
// One pass: a row is read once and held in registers, blocks walk rows in a fixed order with the
// channel sums in registers, and leave them in the workspace, which a second launch adds up in
// order: the same inputs give the same bits.
#include <algorithm>

#include "block_norm.cuh"

namespace swin {

namespace {

using namespace norm;

struct BwdParams {
  const void *y, *dy;
  const __nv_bfloat16 *f, *dh;
  const float *pre_w, *post_w, *gate, *keep;
  void* dx;
  __nv_bfloat16* df;
  float* partial;  // [blocks, kSums, C]
  int rows, C, per_sample;
  bool rms;
  float alpha, eps, inv_c;
};

constexpr int kSums = 4;
constexpr int kMaxBlocks = 2 * 152;

int blocks_of(int64_t rows, const Shape& s) {
  return (int)std::min<int64_t>(kMaxBlocks, (rows + s.rows_per_block - 1) / s.rows_per_block);
}

// d <- r (d - [mean d] - vhat mean(d vhat)): the gradient through a norm.
template <int LANES, int CH>
__device__ __forceinline__ void through_norm(float (&d)[CH][8], const float (&vhat)[CH][8], float r, bool rms,
                                             float inv_c, RowSum<LANES>& sum) {
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s.x += d[j][e];
      s.y = fmaf(d[j][e], vhat[j][e], s.y);
    }
  s = sum(s);
  const float m0 = rms ? 0.0f : s.x * inv_c, m1 = s.y * inv_c;
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) d[j][e] = r * (d[j][e] - fmaf(vhat[j][e], m1, m0));
}

template <typename S, int LANES, int CH>
__global__ void __launch_bounds__(LANES == 0 ? 512 : kThreads) block_norm_bwd_kernel(const BwdParams p) {
  constexpr int kWidth = LANES == 0 ? 1 : LANES * CH * 8;
  __shared__ float2 slots[LANES == 0 ? 32 : 1];
  __shared__ float warp_sums[kThreads / 32][kWidth];
  pdl_launch_dependents();
  pdl_wait();
  RowSum<LANES> sum{slots};
  const int width = LANES == 0 ? blockDim.x : LANES;
  const int lane = LANES == 0 ? threadIdx.x : threadIdx.x % width;
  const int per_block = LANES == 0 ? 1 : kThreads / width;
  int col[CH];
  bool in[CH];
  float acc[kSums][CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    col[j] = (j * width + lane) * 8;
    in[j] = col[j] < p.C;
#pragma unroll
    for (int s = 0; s < kSums; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[s][j][e] = 0.0f;
  }
  for (int64_t row0 = (int64_t)blockIdx.x * per_block; row0 < p.rows; row0 += (int64_t)gridDim.x * per_block) {
    const int64_t own = row0 + (LANES == 0 ? 0 : threadIdx.x / width);
    const bool valid = own < p.rows;
    const int64_t row = valid ? own : p.rows - 1;  // every thread takes part in the sums over the row
    float d[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[j][e] = 0.0f;
      if (p.dy != nullptr && in[j]) load8(static_cast<const S*>(p.dy) + row * p.C + col[j], d[j]);
    }
    if (p.pre_w != nullptr) {
      float v[CH][8], g[CH][8];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = g[j][e] = 0.0f;
        if (in[j]) {
          load8(static_cast<const S*>(p.y) + row * p.C + col[j], v[j]);
          load8(p.dh + row * p.C + col[j], g[j]);
        }
      }
      const float r = normalise<LANES, CH>(v, in, p.rms, p.inv_c, p.eps, sum);
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (!in[j]) continue;
        float w[8];
        load_param8(p.pre_w + col[j], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (valid) {
            acc[0][j][e] = fmaf(g[j][e], v[j][e], acc[0][j][e]);
            acc[1][j][e] += g[j][e];
          }
          g[j][e] *= w[e];
        }
      }
      through_norm<LANES, CH>(g, v, r, p.rms, p.inv_c, sum);
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[j][e] += g[j][e];
    }
    if (valid && p.dx != nullptr) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (!in[j]) continue;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = p.alpha * d[j][e];
        store8(static_cast<S*>(p.dx) + row * p.C + col[j], o);
      }
    }
    if (p.f == nullptr) continue;
    float u[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[j][e] = 0.0f;
      if (in[j]) load8(p.f + row * p.C + col[j], u[j]);
    }
    const float keep = p.keep != nullptr ? p.keep[(unsigned)row / (unsigned)p.per_sample] : 1.0f;
    float r = 1.0f;
    if (p.post_w != nullptr) r = normalise<LANES, CH>(u, in, p.rms, p.inv_c, p.eps, sum);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if (!in[j]) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[j][e] *= keep;
        if (valid) {
          acc[2][j][e] = fmaf(d[j][e], u[j][e], acc[2][j][e]);
          acc[3][j][e] += d[j][e];
        }
      }
      float a[8];
      if (p.gate != nullptr) {
        load_param8(p.gate + col[j], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[j][e] *= a[e];
      }
      if (p.post_w != nullptr) {
        load_param8(p.post_w + col[j], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[j][e] *= a[e];
      }
    }
    if (p.post_w != nullptr) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[j][e] = in[j] ? d[j][e] : 0.0f;
      through_norm<LANES, CH>(d, u, r, p.rms, p.inv_c, sum);
    }
    if (valid)
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (in[j]) store8(p.df + row * p.C + col[j], d[j]);
  }
  // this block's sums
  float* out = p.partial + (int64_t)blockIdx.x * kSums * p.C;
  if constexpr (LANES == 0) {
#pragma unroll
    for (int s = 0; s < kSums; ++s)
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (in[j]) store8(out + (int64_t)s * p.C + col[j], acc[s][j]);
  } else {
#pragma unroll
    for (int s = 0; s < kSums; ++s) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float a = acc[s][j][e];
#pragma unroll
          for (int o = LANES; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
          if ((threadIdx.x & 31) < LANES) warp_sums[threadIdx.x >> 5][col[j] + e] = a;
        }
      __syncthreads();
      for (int c = threadIdx.x; c < p.C; c += kThreads) {
        float a = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) a += warp_sums[w][c];
        out[(int64_t)s * p.C + c] = a;
      }
      __syncthreads();
    }
  }
}

struct ParamGrads {
  const float *post_w, *post_b, *gate;
  float *pre_w_out, *pre_b_out, *post_w_out, *post_b_out, *gate_out;
  bool has_post, accumulate;
};

// The parameter gradients of 32 channels: the blocks' sums, sixteen threads a channel each over every
// sixteenth block, then in order.
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(32 * kSumRows)
    param_grads_kernel(const float* __restrict__ partial, int blocks, int C, const ParamGrads g) {
  __shared__ float part[kSums][kSumRows][32];
  pdl_launch_dependents();
  pdl_wait();
  const int x = threadIdx.x % 32, y = threadIdx.x / 32, c = blockIdx.x * 32 + x;
  float s[kSums] = {};
  if (c < C) {
#pragma unroll 4
    for (int b = y; b < blocks; b += kSumRows) {
#pragma unroll
      for (int k = 0; k < kSums; ++k) s[k] += __ldcg(partial + ((int64_t)b * kSums + k) * C + c);
    }
  }
#pragma unroll
  for (int k = 0; k < kSums; ++k) part[k][y][x] = s[k];
  __syncthreads();
  if (y != 0 || c >= C) return;
#pragma unroll
  for (int k = 0; k < kSums; ++k)
    for (int i = 1; i < kSumRows; ++i) s[k] += part[k][i][x];
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

template <typename S>
cudaError_t launch(const BwdParams& p, const Shape& s, int blocks, cudaStream_t st) {
  const dim3 grid(blocks), block(s.threads);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, block, 0, st, p); };
  switch (s.lanes * 4 + s.chunks) {
    case 4 * 4 + 2: return go(block_norm_bwd_kernel<S, 4, 2>);
    case 4 * 4 + 3: return go(block_norm_bwd_kernel<S, 4, 3>);
    case 8 * 4 + 2: return go(block_norm_bwd_kernel<S, 8, 2>);
    case 8 * 4 + 3: return go(block_norm_bwd_kernel<S, 8, 3>);
    case 16 * 4 + 2: return go(block_norm_bwd_kernel<S, 16, 2>);
    case 16 * 4 + 3: return go(block_norm_bwd_kernel<S, 16, 3>);
    case 32 * 4 + 2: return go(block_norm_bwd_kernel<S, 32, 2>);
    case 32 * 4 + 3: return go(block_norm_bwd_kernel<S, 32, 3>);
    default: return go(block_norm_bwd_kernel<S, 0, 2>);
  }
}

}  // namespace

size_t block_norm_bwd_workspace_bytes(int tokens, int C) {
  return std::max<size_t>(256, (size_t)blocks_of(tokens, shape_of(C)) * kSums * C * 4);
}

cudaError_t block_norm_bwd_launch(const void* y, const void* f, const void* dh, const void* dy, const float* pre_w,
                                  const float* post_w, const float* post_b, const float* gate, const float* keep,
                                  void* dx, void* df, float* dpre_w, float* dpre_b, float* dpost_w, float* dpost_b,
                                  float* dgate, int tokens, int C, int samples, int dtype, int kind, float alpha,
                                  float eps, int accumulate, void* workspace, cudaStream_t st) {
  const Shape s = shape_of(C);
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
  p.alpha = alpha;
  p.eps = eps;
  p.inv_c = 1.0f / (float)C;
  if (tokens > 0) {
    const cudaError_t e = dtype == SWIN_WATTN_FP32 ? launch<float>(p, s, blocks, st) : launch<__nv_bfloat16>(p, s, blocks, st);
    if (e != cudaSuccess) return e;
  }
  ParamGrads g{post_w, post_b, gate, dpre_w, dpre_b, dpost_w, dpost_b, dgate, post_w != nullptr, accumulate != 0};
  if (dpre_w == nullptr && dpre_b == nullptr && dpost_w == nullptr && dpost_b == nullptr && dgate == nullptr)
    return cudaSuccess;
  return launch_pdl(param_grads_kernel, dim3((C + 31) / 32), dim3(32 * kSumRows), 0, st, (const float*)p.partial, blocks, C, g);
}

}  // namespace swin
