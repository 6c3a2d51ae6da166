// The residual sum around a block with its gate and the norms on both sides:
//   u = post(f) or f,   y = alpha x + keep[sample] gate[channel] u,   h = pre(y)
// pre is the norm before the next block, post the one after this block (a res-post-norm block
// has both); either may be absent, and without f the kernel is a plain norm of x.
// One pass: a row is read once, both norms' sums are taken in registers, y and h are written.
// h is normalised from y in fp32, before y is rounded for its store: its one rounding is the one
// to bf16. Bound by memory, 8 bytes an element of bf16 with f; what stood against it was the instructions of a row.
// Two forms:
// * block_norm_kernel: two rows to a group of threads, as many blocks as that takes: fp32 streams, wide rows, few of middling
//   width;
// * block_norm_ring_kernel: resident blocks walk rows, the rows to come on their way through shared memory, the
//   parameters kept there: the others of a bf16 stream.
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
  int stages;  // of the ring: rows of a group in shared memory
  bool rms, vec;
  float alpha, eps, inv_c;
};

// A group takes kRows rows at a time: the parameters, as many bytes of a row as its own in bf16, are read from the
// caches once for both, and one round of sums serves both. (A row at a time, 25088 x 768 with gate took 32.6 us instead of
// 30.3.) One row where a thread has three or four chunks, whose registers for two leave one block on an SM (2400 x 8192: 51
// us, 38 with one).
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

// BLOCKS: of 512 threads that have to fit an SM, which the compiler takes for a limit of registers; 0: none is named.
template <typename S, int LANES, int CH, int BLOCKS = 0>
__global__ void __launch_bounds__(LANES == 0 ? 32 * kMaxWarps : kThreads, BLOCKS) block_norm_kernel(const FwdParams p) {
  __shared__ __align__(8) float slots[LANES == 0 ? 4 * kMaxWarps : 1];
  pdl_launch_dependents();
  pdl_wait();
  RowSum<LANES, kHalves> sum{slots};
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

// ---- rows in turn ------------------------------------------------------------------------

// One row to a group of threads at a time, up to 1536 channels in a warp, so that no barrier stands in a row's way: of
// three chunks a thread and fewer four blocks an SM, of four three, of six two, above one of twelve warps. A row of 768 costs
// half the instructions of block_norm_kernel's, which reads its parameters for two rows and then begins anew.
__host__ __device__ constexpr int ring_threads(int chunks) { return chunks >= 8 ? 384 : 256; }
__host__ __device__ constexpr int ring_blocks(int chunks) { return chunks <= 3 ? 4 : chunks == 4 ? 3 : chunks == 6 ? 2 : 1; }

// Shared bytes of a thread's part of a row: x and, with F, f in bf16.
__host__ __device__ constexpr int ring_bytes(int chunks, bool with_f) { return chunks * kV * (with_f ? 4 : 2); }

// F, POST: whether there are a block's output and a norm behind it.
template <int LANES, int CH, bool F, bool POST>
__global__ void __launch_bounds__(ring_threads(CH), ring_blocks(CH)) block_norm_ring_kernel(const FwdParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  pdl_launch_dependents();
  constexpr int kOwn = ring_threads(CH), kPer = kOwn / LANES, kStride = LANES * kV;
  const int lane = threadIdx.x % LANES, own_row = threadIdx.x / LANES;
  const int64_t step = (int64_t)gridDim.x * kPer;
  RowSum<LANES, kHalves> sum{nullptr};
  // first the parameters, [CH][LANES] each: the norm before the next block, and post and gate in one
  float4* const pre_w = reinterpret_cast<float4*>(smem);
  float4* const pre_b = pre_w + CH * LANES;
  float4* const behind_w = pre_b + CH * LANES;
  float4* const behind_b = behind_w + CH * LANES;
  // then the stages: for each thread CH chunks of x, then of f
  unsigned char* const ring = smem + (F ? 4 : 2) * CH * LANES * 16;
  auto slot = [&](int stage, int k) {
    return reinterpret_cast<uint2*>(ring + stage * (ring_bytes(CH, F) * kOwn)) + k * kOwn + (int)threadIdx.x;
  };
  bool in[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    in[j] = (j * LANES + lane) * kV < p.C;
    if (!in[j])  // chunks outside the row stay zero
      for (int s = 0; s < p.stages; ++s) {
        *slot(s, j) = make_uint2(0, 0);
        if (F) *slot(s, CH + j) = make_uint2(0, 0);
      }
  }
  pdl_wait();
  int64_t row = (int64_t)blockIdx.x * kPer + own_row, ahead = row;  // the row to fetch next
  const int64_t at0 = row * p.C + lane * kV, advance = step * p.C;
  const __nv_bfloat16 *x_next = static_cast<const __nv_bfloat16*>(p.x) + at0, *f_next = p.f + at0;
  auto fetch = [&](int stage) {
    if (ahead < p.rows) {  // (behind the last row the slots keep what they hold; it is not stored)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (!in[j]) continue;
        copy_async<8>(slot(stage, j), x_next + j * kStride);
        if (F) copy_async<8>(slot(stage, CH + j), f_next + j * kStride);
      }
    }
    cp_async_commit();
    ahead += step;
    x_next += advance;
    f_next += advance;
  };
  for (int s = 0; s < p.stages - 1; ++s) fetch(s);
  for (int c = threadIdx.x; c < CH * LANES * kV; c += kOwn) {
    const bool is = c < p.C;
    if (p.pre_w != nullptr) {
      reinterpret_cast<float*>(pre_w)[c] = is ? p.pre_w[c] : 0.0f;
      reinterpret_cast<float*>(pre_b)[c] = is && p.pre_b != nullptr ? p.pre_b[c] : 0.0f;
    }
    if constexpr (F) {
      const float g = is && p.gate != nullptr ? p.gate[c] : 1.0f;
      reinterpret_cast<float*>(behind_w)[c] = POST && is ? p.post_w[c] * g : g;
      reinterpret_cast<float*>(behind_b)[c] = POST && is && p.post_b != nullptr ? p.post_b[c] * g : 0.0f;
    }
  }
  __syncthreads();
  int stage = 0;
  __nv_bfloat16 *y = static_cast<__nv_bfloat16*>(p.y) + at0, *h = p.h + at0;
  for (int64_t row0 = row - own_row; row0 < p.rows; row0 += step, row += step, y += advance, h += advance) {
    fetch(stage == 0 ? p.stages - 1 : stage - 1);
    if (p.stages == 3)
      cp_async_wait<2>();
    else
      cp_async_wait<1>();
    const bool valid = row < p.rows;  // every thread takes part in the sums over the row
    Four v[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) v[j] = unpack4(*slot(stage, j));
    if constexpr (F) {
      Four u[CH];
#pragma unroll
      for (int j = 0; j < CH; ++j) u[j] = unpack4(*slot(stage, CH + j));
      if constexpr (POST) normalise<LANES, CH>(u, in, p.rms, p.inv_c, p.eps, sum);
      const float keep = p.keep != nullptr && valid ? p.keep[(unsigned)row / (unsigned)p.per_sample] : 1.0f;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if constexpr (POST)
          u[j] = fma(u[j], unpack4(behind_w[j * LANES + lane]), unpack4(behind_b[j * LANES + lane]));
        else if (p.gate != nullptr)
          u[j] = mul(u[j], unpack4(behind_w[j * LANES + lane]));
        v[j] = fma(v[j], p.alpha, mul(u[j], keep));
        if (valid && in[j]) store4(y + j * kStride, v[j]);
      }
    }
    if (p.pre_w != nullptr) {
      normalise<LANES, CH>(v, in, p.rms, p.inv_c, p.eps, sum);
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (valid && in[j]) store4(h + j * kStride, fma(v[j], unpack4(pre_w[j * LANES + lane]), unpack4(pre_b[j * LANES + lane])));
    }
    stage = stage == p.stages - 1 ? 0 : stage + 1;
  }
  cp_async_wait_all();
}

template <int LANES, int CH>
cudaError_t launch_ring(FwdParams p, cudaStream_t st) {
  const bool with_f = p.f != nullptr;
  constexpr int kOwn = ring_threads(CH), kBlocks = ring_blocks(CH);
  const int row = ring_bytes(CH, with_f) * kOwn, params = (with_f ? 4 : 2) * CH * LANES * 16, per = kOwn / LANES;
  p.stages = std::min(3, (kMaxSmem / kBlocks - 1024 - params) / row);  // (two at least, of twelve chunks with f)
  const int smem = params + p.stages * row, blocks = (int)std::min<int64_t>(152 * kBlocks, ((int64_t)p.rows + per - 1) / per);
  if (!with_f) return launch_rows<block_norm_ring_kernel<LANES, CH, false, false>>(p, blocks, kOwn, smem, st);
  if (p.post_w == nullptr) return launch_rows<block_norm_ring_kernel<LANES, CH, true, false>>(p, blocks, kOwn, smem, st);
  return launch_rows<block_norm_ring_kernel<LANES, CH, true, true>>(p, blocks, kOwn, smem, st);
}

// A group's lanes and chunks in the ring, of the least capacity, or none: rows of a bf16 stream, up to 384 channels, or up
// to 1536 where there are two rows at least for each group that is resident. (This form and the other, of norm and sum, with
// gate and depth, and with post besides: 100352 x 192 26.2, 26.2, 26.6 us and 29.9, 33.7, 37.9; 1000 x 192 2.2, 2.4, 2.5 and
// 2.6, 3.5, 4.1; 25088 x 768 26.8, 28.2, 28.5 and 26.7, 30.2, 36.8; 4800 x 768 7.0, 7.7, 8.3 and 6.7, 8.2, 10.0; 2500 x 768
// 4.6, 5.0, 5.6 and 3.9, 4.4, 5.4; 12544 x 1536 28.8, 29.7, 31.5 and 27.8, 31.6, 38.4; the norm alone 25088 x 768 15.5 and
// 20.1. Of fp32, 200704 x 192, 74.6, 76.1, 78.8 and 68.9, 70.7, 75.5.)
Shape ring_of(int64_t rows, int C) {
  const int n = C / kV;
  for (int lanes = 4; lanes <= 32; lanes *= 2)
    for (int ch : {2, 3, 4, 6, 8, 12})
      if (n <= lanes * ch && (ch <= 3 || lanes == 32)) {
        const int per = ring_threads(ch) / lanes;
        if (ch > 3 && rows < (int64_t)2 * 152 * ring_blocks(ch) * per) return {};
        return {lanes, ch, ring_threads(ch), per};
      }
  return {};
}

template <typename S>
cudaError_t launch(const FwdParams& p, cudaStream_t st) {
  if constexpr (sizeof(S) == 2) {
    const Shape r = ring_of(p.rows, p.C);
    switch (r.lanes * 16 + r.chunks) {
      case 4 * 16 + 2: return launch_ring<4, 2>(p, st);
      case 4 * 16 + 3: return launch_ring<4, 3>(p, st);
      case 8 * 16 + 2: return launch_ring<8, 2>(p, st);
      case 8 * 16 + 3: return launch_ring<8, 3>(p, st);
      case 16 * 16 + 2: return launch_ring<16, 2>(p, st);
      case 16 * 16 + 3: return launch_ring<16, 3>(p, st);
      case 32 * 16 + 2: return launch_ring<32, 2>(p, st);
      case 32 * 16 + 3: return launch_ring<32, 3>(p, st);
      case 32 * 16 + 4: return launch_ring<32, 4>(p, st);
      case 32 * 16 + 6: return launch_ring<32, 6>(p, st);
      case 32 * 16 + 8: return launch_ring<32, 8>(p, st);
      case 32 * 16 + 12: return launch_ring<32, 12>(p, st);
      default: break;
    }
  }
  const Shape s = shape_of(p.C);
  const int per_block = s.rows_per_block * rows_of(s.lanes, s.chunks);
  const dim3 grid((unsigned)(((int64_t)p.rows + per_block - 1) / per_block)), block(s.threads);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, block, 0, st, p); };
  if constexpr (sizeof(S) == 4) {  // (in bf16 these walk)
    switch (s.lanes * 8 + s.chunks) {
      case 4 * 8 + 2: return go(block_norm_kernel<S, 4, 2>);
      case 4 * 8 + 3: return go(block_norm_kernel<S, 4, 3>);
      case 8 * 8 + 2: return go(block_norm_kernel<S, 8, 2>);
      case 8 * 8 + 3: return go(block_norm_kernel<S, 8, 3>);
      case 16 * 8 + 2: return go(block_norm_kernel<S, 16, 2>);
      case 16 * 8 + 3: return go(block_norm_kernel<S, 16, 3>);
      case 32 * 8 + 2: return go(block_norm_kernel<S, 32, 2>);
      case 32 * 8 + 3: return go(block_norm_kernel<S, 32, 3>);
      default: break;
    }
  }
  switch (s.chunks) {
    // 52 registers instead of 59 for fp32 and above 1536 channels (8000 x 2304 with gate and depth 32.4 -> 29.0 us, 12544 x 1536
    // fp32 with post besides 40.5 -> 39.0; but 2500 x 768 of bf16 4.1 -> 4.6)
    case 2: return sizeof(S) == 4 || p.C > 1536 ? go(block_norm_kernel<S, 0, 2, 2>) : go(block_norm_kernel<S, 0, 2>);
    case 3: return go(block_norm_kernel<S, 0, 3>);
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
