// A stack of weight updates brought near orthogonal by Newton-Schulz products. Per matrix
// G (rows x cols):
//   X = G / (|G|_F + eps);   `steps` times:  A = X X^T,  X <- (a I + b A + c A^2) X;
//   out = scale X                  (A = X^T X and X <- X (a I + b A + c A^2) when rows > cols)
// with (a, b, c) = (3.4445, -4.7750, 2.0315): each step applies the odd quintic
// a s + b s^3 + c s^5 to every singular value s, which takes (0, 1] towards [0.7, 1.2] and
// stays below 1.21, so U V^T of G = U S V^T is approached with every singular value within
// that band, without a decomposition.
//
// All products run on the engine of product.cuh. Nothing is transposed: for wide matrices
// the Gram product reads X K-major twice and the update reads X MN-major; for tall ones the
// Gram product reads X MN-major twice and the update reads it K-major; A and the
// polynomial B = a I + b A + c A^2 are symmetric.
//
// Operands are fp16, not bf16: the entries of X, A and B are bounded (|X| <= 1.21,
// |A| <= 1.45, |B| < 16), so the exponent range of bf16 is not needed and its 8 significant
// bits cost eight times the error. X is held in two parts, its rounding and what that leaves, and
// the update's product walks K once for each (why: orthogonalize.cuh, with the diagonals of A
// and B); A is made of the larger part, whose rounding there does what A's own does. Before the
// rounding to bf16 (1.7e-3 by itself, relative 2-norm) five steps end 0.5e-3 to 1.7e-3 from the
// 64-bit result, over spectra from flat to 1 / k^2, halves a thousandfold apart and ranks from
// 1. A and B are kept times 2^8, which leaves the largest B a tenth of the largest fp16, X times
// 2^14, which leaves the smaller part of a typical entry (1 / sqrt(rows cols) = 3e-4 at
// 1536 x 6144) some ten bits. Products are accumulated in fp32.
//
// A and B are symmetric. Where it is estimated to pay, only the tiles on and below their
// diagonals are computed, and stored twice (product.cuh): two 1536 x 6144 take 72 tiles of 256 x 160
// in one round of the pairs instead of 72 of 256 x 256, and less power.
//
// Measured on one GB300, graph of calls: two 1536 x 6144 650 us, of which the second part of X takes
// some 43 us a step (441 us on the same card with X in one part), bound by the tensor cores; eight
// 2048 x 512 192 us (154), bound by the chain of seventeen dependent launches.
// (With X in one part: all tiles of A and B 451 us where half of them took 418; one epilogue for
// all three products, which tells them apart as it runs, 169 us for the stack where three took 151.)
#include "orthogonalize.cuh"
#include "product.cuh"

namespace swin {

bool orthogonalize_small_applies(int rows, int cols);
cudaError_t orthogonalize_small_launch(const void* g, void* out, int count, int rows, int cols, int dtype, int steps,
                                       float eps, float scale, int* status, cudaStream_t st);

namespace {

using prod::Matrix;
using prod::Params;
using prod::Tiling;

constexpr CUtensorMapDataType kF16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
constexpr CUtensorMapDataType kF32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

constexpr int kNormThreads = 256;
constexpr int kNormBlocks = 256;  // partial sums per matrix at most

// Blocks per matrix: four per SM over the stack, of 2048 elements each at least.
int norm_blocks(int64_t elements, int count) {
  return (int)std::max<int64_t>(1, std::min<int64_t>({kNormBlocks, (elements + 2047) / 2048, (4 * prod::kSms + count - 1) / count}));
}

// The sum over the block, in every thread.
__device__ __forceinline__ Squares block_sum(const Squares& s) {
  __shared__ Squares part[kNormThreads / 32];
  const Squares w = warp_sum(s);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = w;
  __syncthreads();
  Squares b = part[0];
  for (int w = 1; w < kNormThreads / 32; ++w) add(b, part[w]);
  return b;
}
__device__ __forceinline__ float block_sum(float s) {
  __shared__ float part[kNormThreads / 32];
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = part[0];
  for (int w = 1; w < kNormThreads / 32; ++w) s += part[w];
  return s;
}

// Sum of squares of a block's share of one matrix. `vec`: every matrix starts on a 16-byte
// boundary and holds a multiple of eight elements, which are then read eight at a time, four
// such reads in flight.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_partial_kernel(const T* __restrict__ g, int64_t elements, bool vec,
                                                                    Squares* __restrict__ partial) {
  pdl_launch_dependents();
  pdl_wait();
  const T* x = g + (int64_t)blockIdx.y * elements;
  const int64_t first = (int64_t)blockIdx.x * kNormThreads + threadIdx.x, stride = (int64_t)gridDim.x * kNormThreads;
  float2 plain = make_float2(0.0f, 0.0f);
  if (vec) {
    const int64_t n8 = elements / 8;
    int64_t i = first;
    for (; i + 3 * stride < n8; i += 4 * stride) {
      float v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) load8(x + (i + u * stride) * 8, v[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) add_plain(v[u], plain);
    }
    for (; i < n8; i += stride) {
      float v[8];
      load8(x + i * 8, v);
      add_plain(v, plain);
    }
  } else {
    for (int64_t i = first; i < elements; i += stride) {
      const float v = load_f32(x + i);
      plain.x = fmaf(v, v, plain.x);
    }
  }
  Squares sum{block_sum(plain.x + plain.y), 0.0f, 0.0f};
  if (!plain_sum_holds(sum.mid)) {
    // the same share, an element at a time
    const int64_t per = vec ? 8 : 1;
    sum.mid = 0.0f;
    for (int64_t i = first; i < elements / per; i += stride)
      for (int64_t e = 0; e < per; ++e) add_square(load_f32(x + i * per + e), sum);
    sum = block_sum(sum);
  }
  if (threadIdx.x == 0) partial[blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// X = G / (|G| + eps), times 2^14, in two fp16 parts, of `rows` rows of ld elements each.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) normalize_kernel(const T* __restrict__ g, int rows, int cols, int ld,
                                                                 bool vec, const Squares* __restrict__ partial,
                                                                 int n_partial, float eps, __half* __restrict__ x) {
  pdl_launch_dependents();
  pdl_wait();
  Squares sum{};
  if ((int)threadIdx.x < n_partial) sum = partial[blockIdx.y * n_partial + threadIdx.x];
  const Inverse k = inverse_of(block_sum(sum), eps);
  const int64_t elements = (int64_t)rows * cols;
  const T* gm = g + (int64_t)blockIdx.y * elements;
  __half* xm = x + (int64_t)blockIdx.y * 2 * rows * ld;
  __half* low = xm + (int64_t)rows * ld;
  if (vec && ld == cols) {
    const int64_t n8 = elements / 8, stride = (int64_t)gridDim.x * kNormThreads;
#pragma unroll 4
    for (int64_t i = (int64_t)blockIdx.x * kNormThreads + threadIdx.x; i < n8; i += stride) {
      float v[8];
      load8(gm + i * 8, v);
      uint32_t o[4], r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) two_parts(make_float2(v[2 * e] * k.pre * k.inv, v[2 * e + 1] * k.pre * k.inv), o[e], r[e]);
      reinterpret_cast<uint4*>(xm)[i] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4*>(low)[i] = make_uint4(r[0], r[1], r[2], r[3]);
    }
  } else {
    const int wpb = kNormThreads / 32, lane = threadIdx.x & 31;
    for (int r = blockIdx.x * wpb + (threadIdx.x >> 5); r < rows; r += gridDim.x * wpb)
      for (int c = lane; c < cols; c += 32) {
        const float v = load_f32(gm + (int64_t)r * cols + c) * k.pre * k.inv;
        const __half h = __float2half_rn(v);
        xm[(int64_t)r * ld + c] = h;
        low[(int64_t)r * ld + c] = __float2half_rn(v - __half2float(h));
      }
  }
}

// A' = sum over the splits of the Gram product's parts, less mu on the diagonal: four columns a
// thread, all parts' reads in flight (they are in L2). Rows have ld elements, of parts and result.
constexpr int kSumThreads = 128;
__global__ void __launch_bounds__(kSumThreads) gram_sum_kernel(const float* __restrict__ part, int splits, int m, int ld,
                                                               float mu, __half* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x * kSumThreads + threadIdx.x;  // four columns of the matrix
  if (i >= m * (ld / 4)) return;
  const int64_t size = (int64_t)m * ld;
  const float4* p = reinterpret_cast<const float4*>(part + blockIdx.y * splits * size) + i;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    const float4 a = __ldcg(p + s * (size / 4));
    v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
  }
  const int r = i / (ld / 4), c = i % (ld / 4) * 4;
  constexpr float k = kScale / (kScaleX * kScaleX);
  const float d = -mu * kScale;
  reinterpret_cast<uint2*>(out + blockIdx.y * size)[i] =
      make_uint2(prod::pack_f16(fmaf(v.x, k, r == c ? d : 0.0f), fmaf(v.y, k, r == c + 1 ? d : 0.0f)),
                 prod::pack_f16(fmaf(v.z, k, r == c + 2 ? d : 0.0f), fmaf(v.w, k, r == c + 3 ? d : 0.0f)));
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
int round8(int n) { return (n + 7) & ~7; }

// The Gram product, over the longer side. Where that is long and its tiles are few, it is split
// into parts and their sum is a launch of its own (two 70 x 5497, three steps: 109 us whole, 65 us in
// parts; 512 x 2048, five steps: 100 and 90 us; 300 x 900: 72 and 76 us). The 500 clocks keep ties whole.
constexpr int kMaxGramSplits = 16;
Tiling gram_tiling(int count, int rows, int cols) {
  const int m = std::min(rows, cols), n = std::max(rows, cols);
  const bool tall = rows > cols;
  const Tiling whole = prod::choose_tiling(m, m, n, count, tall, 1, false, true);
  const Tiling parts = prod::choose_tiling(m, m, n, count, tall, kMaxGramSplits, false);
  return parts.splits > 1 && prod::tiling_cost(parts, m, m, count, tall, false) + 500.0 <
                                 prod::tiling_cost(whole, m, m, count, tall, false)
             ? parts
             : whole;
}

// Workspace: two copies of X in two parts, A, B, the factors of B's diagonal, the partial sums of squares, the
// parts of the Gram product.
struct Layout {
  int m, ldx, lda, ld_gain;
  size_t x_bytes, a_bytes, gain_bytes, partial_bytes, total;
};
Layout layout(int count, int rows, int cols) {
  Layout l;
  l.m = std::min(rows, cols);
  l.ldx = round8(cols);
  l.lda = round8(l.m);
  l.x_bytes = align256((size_t)count * 2 * rows * l.ldx * 2);
  l.a_bytes = align256((size_t)count * l.m * l.lda * 2);
  l.ld_gain = (l.m + 31) & ~31;
  l.gain_bytes = align256((size_t)count * l.ld_gain * sizeof(float));
  l.partial_bytes = align256((size_t)count * kNormBlocks * sizeof(Squares));
  const int splits = gram_tiling(count, rows, cols).splits;
  l.total = 2 * l.x_bytes + 2 * l.a_bytes + l.gain_bytes + l.partial_bytes +
            (splits > 1 ? align256((size_t)count * splits * l.m * l.lda * 4) : 0);
  return l;
}

template <typename T>
cudaError_t normalize(const T* g, int count, int rows, int cols, float eps, Squares* partial, __half* x, int ld,
                      cudaStream_t st) {
  const int64_t elements = (int64_t)rows * cols;
  const int nb = norm_blocks(elements, count);
  const bool vec = elements % 8 == 0 && reinterpret_cast<uintptr_t>(g) % 16 == 0;
  cudaError_t e = launch_pdl(norm_partial_kernel<T>, dim3(nb, count), dim3(kNormThreads), 0, st, g, elements, vec, partial);
  if (e != cudaSuccess) return e;
  return launch_pdl(normalize_kernel<T>, dim3(nb, count), dim3(kNormThreads), 0, st, g, rows, cols, ld, vec,
                    (const Squares*)partial, nb, eps, x);
}

}  // namespace

size_t orthogonalize_workspace_bytes(int count, int rows, int cols) {
  return orthogonalize_small_applies(rows, cols) ? 256 : layout(count, rows, cols).total;
}
int orthogonalize_launches(int count, int rows, int cols, int steps) {
  return orthogonalize_small_applies(rows, cols) ? 1 : 2 + (gram_tiling(count, rows, cols).splits > 1 ? 4 : 3) * steps;
}

cudaError_t orthogonalize_launch(const void* g, void* out, int count, int rows, int cols, int dtype, int steps,
                                 float eps, float scale, void* workspace, int* status, cudaStream_t st) {
  if (orthogonalize_small_applies(rows, cols))
    return orthogonalize_small_launch(g, out, count, rows, cols, dtype, steps, eps, scale, status, st);
  const Layout l = layout(count, rows, cols);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  __half* x[2] = {reinterpret_cast<__half*>(ws), reinterpret_cast<__half*>(ws + l.x_bytes)};
  __half* gram = reinterpret_cast<__half*>(ws + 2 * l.x_bytes);
  __half* poly = reinterpret_cast<__half*>(ws + 2 * l.x_bytes + l.a_bytes);
  float* gain = reinterpret_cast<float*>(ws + 2 * l.x_bytes + 2 * l.a_bytes);
  Squares* partial = reinterpret_cast<Squares*>(ws + 2 * l.x_bytes + 2 * l.a_bytes + l.gain_bytes);
  float* parts = reinterpret_cast<float*>(ws + 2 * l.x_bytes + 2 * l.a_bytes + l.gain_bytes + l.partial_bytes);
  cudaError_t e = dtype == SWIN_WATTN_FP32
                      ? normalize(static_cast<const float*>(g), count, rows, cols, eps, partial, x[0], l.ldx, st)
                      : normalize(static_cast<const __nv_bfloat16*>(g), count, rows, cols, eps, partial, x[0], l.ldx, st);
  const bool tall = rows > cols;
  const int m = l.m, n = std::max(rows, cols);
  const Tiling t_gram = gram_tiling(count, rows, cols);
  const Tiling t_poly = prod::choose_tiling(m, m, m, count, false, 1, false, true);
  const int part_chunks = (m + prod::kKC - 1) / prod::kKC;
  const Tiling t_step = prod::choose_tiling(rows, cols, 2 * part_chunks * prod::kKC, count, !tall, 1, false);
  const Matrix A{gram, m, m, l.lda, (int64_t)m * l.lda}, B{poly, m, m, l.lda, (int64_t)m * l.lda};
  const bool direct = cols % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  float mu = first_shift(m);
  for (int s = 0; s < steps && e == cudaSuccess; ++s, mu = next_shift(mu)) {
    const NsStep k = ns_step(mu);
    // X in both parts, and its larger part alone, of which A is made
    const Matrix X{x[s & 1], rows, cols, l.ldx, (int64_t)rows * l.ldx, 2}, H{x[s & 1], rows, cols, l.ldx, (int64_t)2 * rows * l.ldx};
    Matrix Y{x[(s + 1) & 1], rows, cols, l.ldx, (int64_t)rows * l.ldx, 2};
    Params p{};
    p.status = status;
    p.M = p.N = m;
    p.alpha = kScale / (kScaleX * kScaleX);  // (2^14 X)(2^14 X)^T = 2^28 A -> 2^8 (A - mu I)
    p.diag = -k.mu * (kScaleX * kScaleX);
    prod::Extra none;
    if (t_gram.splits > 1) {
      const Matrix P{parts, m, m, l.lda, (int64_t)m * l.lda};
      e = tall ? prod::launch_product<true, true, prod::kEpiGrad32>(t_gram, p, H, H, P, count, kF16, kF32, none, st)
               : prod::launch_product<false, false, prod::kEpiGrad32>(t_gram, p, H, H, P, count, kF16, kF32, none, st);
      if (e == cudaSuccess)
        e = launch_pdl(gram_sum_kernel, dim3((m * (l.lda / 4) + kSumThreads - 1) / kSumThreads, count), dim3(kSumThreads), 0,
                       st, (const float*)parts, t_gram.splits, m, l.lda, k.mu, gram);
    } else {
      e = tall ? prod::launch_product<true, true, prod::kEpiGram>(t_gram, p, H, H, A, count, kF16, kF16, none, st)
               : prod::launch_product<false, false, prod::kEpiGram>(t_gram, p, H, H, A, count, kF16, kF16, none, st);
    }
    if (e != cudaSuccess) return e;
    p.alpha = kNsC / kScale;
    p.beta = k.b;
    p.diag = k.e * (kScale * kScale / kNsC);
    p.gain = gain;
    p.gain_ld = l.ld_gain;
    prod::Extra with_a;
    with_a.aux = &A;
    e = prod::launch_product<false, false, prod::kEpiPoly>(t_poly, p, A, A, B, count, kF16, kF16, with_a, st);
    if (e != cudaSuccess) return e;
    Params q{};
    q.status = status;
    q.M = rows;
    q.N = cols;
    q.alpha = 1.0f / kScale;
    q.gain = gain;
    q.gain_ld = l.ld_gain;
    q.gain_rows = !tall;
    q.part_chunks = part_chunks;
    CUtensorMapDataType out_type = kF16;
    if (s == steps - 1) {
      q.alpha = scale / (kScale * kScaleX);
      q.to_bf16 = true;
      out_type = kBf16;
      Y = Matrix{out, rows, cols, cols, (int64_t)rows * cols};
      if (!direct) q.raw_out = static_cast<__nv_bfloat16*>(out);
    }
    e = tall ? prod::launch_product<false, false, prod::kEpiUpdate>(t_step, q, X, B, Y, count, kF16, out_type, none, st)
             : prod::launch_product<false, true, prod::kEpiUpdate>(t_step, q, B, X, Y, count, kF16, out_type, none, st);
  }
  return e;
}

}  // namespace swin
