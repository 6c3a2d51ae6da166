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
#pragma once

#include "block_norm.cuh"

namespace swin {

struct NormBwdParams {
  const void *y, *dy;
  const __nv_bfloat16 *f, *dh;
  const float *pre_w, *post_w, *gate, *keep;
  void* dx;
  __nv_bfloat16* df;
  float* partial;  // [blocks, kSums, C]
  int rows, C, per_sample;
  int stages;  // rows of a group in shared memory: one in use, the others (two; of wide rows one, of fp32 ones above 6144
               // channels none) on their way
  bool rms;
  float alpha, eps, inv_c;
};

namespace {

using namespace norm;
using BwdParams = NormBwdParams;


constexpr int kSums = 4;

constexpr int kThreads = 256;  // of a block of groups that lie in warps

// Of the least capacity: two or three chunks in a warp, four or six in the widest one (a row costs a warp some 250
// instructions whatever it holds, and a block's warps a barrier for each sum besides: 25088 tokens of 768 channels in a
// block of 96 threads 82 us without a norm behind, in a warp 46); then blocks of 4, 8 or 16 warps with two or three chunks,
// above 6144 channels four. With up to 128 registers a thread four warps fit each quarter of an SM, 16 in all, which
// blocks of six or nine warps do not fill (8363 x 2304 in blocks of 288 threads 73 us, with a norm behind 94; 256: 56, 70).
// 12544 x 1536 takes 60 us in blocks of 256 threads, 69 of 128 with three chunks; with a norm behind 80 and 69.
Shape shape_of(int C, bool post) {
  const int n = C / kV;
  for (int lanes = 4; lanes <= 32; lanes *= 2)
    for (int ch : {2, 3, 4, 6})
      if (n <= lanes * ch && (ch <= 3 || lanes == 32)) return {lanes, ch, kThreads, kThreads / lanes};
  for (int threads = 128; threads <= 32 * kMaxWarps; threads *= 2)
    for (int ch = 2; ch <= 3; ++ch)
      if (n <= threads * ch && (threads > 128 || ch == 2 || post)) return {0, ch, threads, 1};
  return {0, 4, 32 * kMaxWarps, 1};
}

// Blocks, and so the channel sums that each leaves: as many as are resident on 152 SMs by their registers.
int blocks_of(int64_t rows, const Shape& s) {
  const int per_sm = s.lanes != 0 ? (s.chunks >= 4 ? 1 : 2) : 32 * kMaxWarps / s.threads;
  return (int)std::min<int64_t>(152 * per_sm, (rows + s.rows_per_block - 1) / s.rows_per_block);
}

// The gradient through a norm: r (g - [mean g] - vhat mean(g vhat)) + more, into g. Chunks outside the row hold zeros and
// are left zero.
template <int LANES, int CH, int FORM>
__device__ __forceinline__ void through_norm(Four (&g)[CH], const Four (&vhat)[CH], const Four (&more)[CH],
                                             const bool (&in)[CH], float r, bool rms, float inv_c, RowSum<LANES, FORM>& sum) {
  Four a = g[0], b = mul(g[0], vhat[0]);
#pragma unroll
  for (int j = 1; j < CH; ++j) {
    a = add(a, g[j]);
    b = fma(g[j], vhat[j], b);
  }
  const float2 sa = __fadd2_rn(a.p[0], a.p[1]), sb = __fadd2_rn(b.p[0], b.p[1]);
  const float2 s = sum(make_float2(sa.x + sa.y, sb.x + sb.y));
  const float c0 = rms ? 0.0f : -r * (s.x * inv_c), c1 = -r * (s.y * inv_c);
#pragma unroll
  for (int j = 0; j < CH; ++j) g[j] = fma(g[j], r, fma(vhat[j], c1, add(more[j], in[j] ? c0 : 0.0f)));
}

// Shared bytes of a thread's part of a row: y and dy of the stream's type, dh and f; and of the parameters, those
// of the norm before and the product of those behind.
template <typename S>
__host__ __device__ constexpr int row_bytes(int chunks) {
  return chunks * kV * (2 * (int)sizeof(S) + 4);
}
__host__ __device__ constexpr int param_bytes(int chunks) { return 2 * chunks * kV * 4; }

// PRE, POST: whether there is a norm before and after (the branches' registers and both norms' sums taken together
// are worth kernels of their own).
template <typename S, int LANES, int CH, bool PRE, bool POST>
__global__ void __launch_bounds__(LANES == 0 ? 32 * kMaxWarps : kThreads, LANES == 0 || CH >= 4 ? 1 : 2)
    block_norm_bwd_kernel(const BwdParams p) {
  using RawS = typename Raw<S>::T;
  constexpr int kWidth = LANES * CH * kV;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(8) float slots[LANES == 0 ? 4 * kMaxWarps : 1];
  pdl_launch_dependents();
  const int threads = LANES == 0 ? blockDim.x : kThreads, width = LANES == 0 ? threads : LANES;
  const int lane = LANES == 0 ? threadIdx.x : threadIdx.x % width;
  const int per_block = LANES == 0 ? 1 : kThreads / width, own_row = LANES == 0 ? 0 : threadIdx.x / width;
  const int64_t step = (int64_t)gridDim.x * per_block;
  RowSum<LANES, PRE && POST ? kEven : kWhole> sum{slots};
  // first the parameters of the row's channels, zeros outside it
  float4* const pre_w = reinterpret_cast<float4*>(smem);  // [CH][width]
  float4* const behind = pre_w + CH * width;
  unsigned char* const ring = smem + 2 * CH * width * 16;
  // a stage: for each thread CH chunks of y, then of dy, then of dh, then of f
  auto stream_slot = [&](int stage, int k) {
    return reinterpret_cast<RawS*>(ring + stage * (row_bytes<S>(CH) * threads)) + k * threads + (int)threadIdx.x;
  };
  auto half_slot = [&](int stage, int k) {
    return reinterpret_cast<uint2*>(ring + stage * (row_bytes<S>(CH) * threads) + 2 * CH * threads * (int)sizeof(RawS)) +
           k * threads + (int)threadIdx.x;
  };
  bool in[CH];
  Four acc[kSums][CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    in[j] = (LANES == 0 && j < CH - 1) || (j * width + lane) * kV < p.C;  // (of a block's chunks only the last may end early)
#pragma unroll
    for (int s = 0; s < kSums; ++s) acc[s][j] = zeros();
    if (!in[j])  // chunks outside the row stay zero
      for (int s = 0; s < p.stages; ++s) {
        *stream_slot(s, j) = *stream_slot(s, CH + j) = RawS{};
        *half_slot(s, j) = *half_slot(s, CH + j) = make_uint2(0, 0);
      }
  }
  pdl_wait();
  // the rows to fetch next
  int64_t ahead = (int64_t)blockIdx.x * per_block + own_row;
  const int64_t at0 = ahead * p.C + lane * kV, advance = step * p.C;
  const S *y_next = static_cast<const S*>(p.y) + at0, *dy_next = static_cast<const S*>(p.dy) + at0;
  const __nv_bfloat16 *dh_next = p.dh + at0, *f_next = p.f + at0;
  const int stride = width * kV;
  auto fetch = [&](int stage) {
    if (ahead < p.rows) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (!in[j]) continue;
        if (PRE) copy_async<sizeof(RawS)>(stream_slot(stage, j), y_next + j * stride);
        if (PRE) copy_async<8>(half_slot(stage, j), dh_next + j * stride);
        if (p.dy != nullptr) copy_async<sizeof(RawS)>(stream_slot(stage, CH + j), dy_next + j * stride);
        if (POST || p.f != nullptr) copy_async<8>(half_slot(stage, CH + j), f_next + j * stride);
      }
    } else {  // behind the last row: zeros, which add nothing to any sum
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        *stream_slot(stage, j) = *stream_slot(stage, CH + j) = RawS{};
        *half_slot(stage, j) = *half_slot(stage, CH + j) = make_uint2(0, 0);
      }
    }
    cp_async_commit();
    ahead += step;
    y_next += advance;
    dy_next += advance;
    dh_next += advance;
    f_next += advance;
  };
  for (int s = 0; s < p.stages - 1; ++s) fetch(s);
  for (int c = threadIdx.x; c < CH * width * kV; c += threads) {
    float a = 0.0f, b = 0.0f;
    if (c < p.C) {
      if (PRE) a = p.pre_w[c];
      b = (p.gate != nullptr ? p.gate[c] : 1.0f) * (POST ? p.post_w[c] : 1.0f);
    }
    reinterpret_cast<float*>(pre_w)[c] = a;
    reinterpret_cast<float*>(behind)[c] = b;
  }
  __syncthreads();
  const bool scaled = POST || p.gate != nullptr;
  int stage = 0;
  S* dx = static_cast<S*>(p.dx) + at0;
  __nv_bfloat16* df = p.df + at0;
  int64_t row = (int64_t)blockIdx.x * per_block + own_row;
  for (int64_t row0 = row - own_row; row0 < p.rows; row0 += step, row += step, dx += advance, df += advance) {
    fetch(stage == 0 ? p.stages - 1 : stage - 1);
    if (p.stages == 3)
      cp_async_wait<2>();
    else if (p.stages == 2)
      cp_async_wait<1>();
    else
      cp_async_wait<0>();
    const bool valid = row < p.rows;  // every thread takes part in the sums over the row
    Four v[CH], u[CH];  // normalised rows of y and f
    float2 r = make_float2(1.0f, 1.0f);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if (PRE) v[j] = unpack4(*stream_slot(stage, j));
      u[j] = POST || p.f != nullptr ? unpack4(*half_slot(stage, CH + j)) : zeros();
    }
    if constexpr (PRE && POST) {
      r = normalise_both<LANES, CH>(v, u, in, p.rms, p.inv_c, p.eps, sum);
    } else {
      if constexpr (PRE) r.x = normalise<LANES, CH>(v, in, p.rms, p.inv_c, p.eps, sum);
      if constexpr (POST) r.y = normalise<LANES, CH>(u, in, p.rms, p.inv_c, p.eps, sum);
    }
    Four d[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) d[j] = p.dy != nullptr ? unpack4(*stream_slot(stage, CH + j)) : zeros();
    if constexpr (PRE) {
      Four g[CH];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        g[j] = unpack4(*half_slot(stage, j));
        acc[0][j] = fma(g[j], v[j], acc[0][j]);
        acc[1][j] = add(g[j], acc[1][j]);
        g[j] = mul(g[j], unpack4(pre_w[j * width + lane]));
      }
      through_norm<LANES, CH>(g, v, d, in, r.x, p.rms, p.inv_c, sum);
#pragma unroll
      for (int j = 0; j < CH; ++j) d[j] = g[j];
    }
    if (valid) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (in[j]) store4(dx + j * stride, p.alpha == 1.0f ? d[j] : mul(d[j], p.alpha));
    }
    if (POST || p.f != nullptr) {
      if (p.keep != nullptr) {
        const float keep = valid ? p.keep[(unsigned)row / (unsigned)p.per_sample] : 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) d[j] = mul(d[j], keep);
      }
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        acc[2][j] = fma(d[j], u[j], acc[2][j]);
        if (POST) acc[3][j] = add(d[j], acc[3][j]);
        if (scaled) d[j] = mul(d[j], unpack4(behind[j * width + lane]));
      }
      if constexpr (POST) {
        Four none[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) none[j] = zeros();
        through_norm<LANES, CH>(d, u, none, in, r.y, p.rms, p.inv_c, sum);
      }
      if (valid) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
          if (in[j]) store4(df + j * stride, d[j]);
      }
    }
    stage = stage == p.stages - 1 ? 0 : stage + 1;
  }
  cp_async_wait_all();
  // this block's sums
  float* out = p.partial + (int64_t)blockIdx.x * kSums * p.C;
  if constexpr (LANES == 0) {
#pragma unroll
    for (int s = 0; s < kSums; ++s)
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (in[j]) store4(out + (int64_t)s * p.C + (j * width + lane) * kV, acc[s][j]);
  } else {
    float* warp_sums = reinterpret_cast<float*>(ring);  // [warps][kWidth], over the rows
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSums; ++s) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 a = acc[s][j].p[i];
#pragma unroll
          for (int o = LANES; o < 32; o <<= 1) {
            a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
            a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
          }
          if ((threadIdx.x & 31) < LANES)
            *reinterpret_cast<float2*>(warp_sums + (threadIdx.x >> 5) * kWidth + (j * LANES + lane) * kV + 2 * i) = a;
        }
      __syncthreads();
      for (int c = threadIdx.x; c < p.C; c += kThreads) {
        float a = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) a += warp_sums[w * kWidth + c];
        out[(int64_t)s * p.C + c] = a;
      }
      __syncthreads();
    }
  }
}

template <typename S, bool PRE, bool POST>
cudaError_t launch(BwdParams p, const Shape& s, int blocks, cudaStream_t st) {
  // (two stages hold the warps' sums, four bytes a thread's channel, in each shape)
  const int row = row_bytes<S>(s.chunks) * s.threads, params = param_bytes(s.chunks) * (s.lanes != 0 ? s.lanes : s.threads);
  const int resident = (blocks + 151) / 152;
  p.stages = std::min(3, (kMaxSmem / resident - 1024 - params) / row);
  const int smem = params + p.stages * row;
  switch (s.lanes * 8 + s.chunks) {
    case 4 * 8 + 2: return launch_rows<block_norm_bwd_kernel<S, 4, 2, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 4 * 8 + 3: return launch_rows<block_norm_bwd_kernel<S, 4, 3, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 8 * 8 + 2: return launch_rows<block_norm_bwd_kernel<S, 8, 2, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 8 * 8 + 3: return launch_rows<block_norm_bwd_kernel<S, 8, 3, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 16 * 8 + 2: return launch_rows<block_norm_bwd_kernel<S, 16, 2, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 16 * 8 + 3: return launch_rows<block_norm_bwd_kernel<S, 16, 3, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 32 * 8 + 2: return launch_rows<block_norm_bwd_kernel<S, 32, 2, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 32 * 8 + 3: return launch_rows<block_norm_bwd_kernel<S, 32, 3, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 32 * 8 + 4: return launch_rows<block_norm_bwd_kernel<S, 32, 4, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 32 * 8 + 6: return launch_rows<block_norm_bwd_kernel<S, 32, 6, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 0 * 8 + 2: return launch_rows<block_norm_bwd_kernel<S, 0, 2, PRE, POST>>(p, blocks, s.threads, smem, st);
    case 0 * 8 + 3: return launch_rows<block_norm_bwd_kernel<S, 0, 3, PRE, POST>>(p, blocks, s.threads, smem, st);
    default: return launch_rows<block_norm_bwd_kernel<S, 0, 4, PRE, POST>>(p, blocks, s.threads, smem, st);
  }
}

template <typename S>
cudaError_t launch(const BwdParams& p, const Shape& s, int blocks, cudaStream_t st) {
  if (p.pre_w != nullptr) return p.post_w != nullptr ? launch<S, true, true>(p, s, blocks, st) : launch<S, true, false>(p, s, blocks, st);
  return p.post_w != nullptr ? launch<S, false, true>(p, s, blocks, st) : launch<S, false, false>(p, s, blocks, st);
}

}  // namespace
}  // namespace swin
