// The products of a block's MLP and their gradients, on the product engine (product.cuh):
//   linear            y  = residual + act(x W^T + b),  pre = x W^T + b   (x [T, K], W [N, K])
//   linear_bwd_data   dx = (dy W) * act'(pre)
//   linear_bwd_weight dW = [dW +] dy^T x,  db = [db +] sum over the tokens of dy
// The operands are read as they lie: in dy W the weight is contracted along its rows, in
// dy^T x both operands are, and the tensor core takes them MN-major.
//
// linear_bwd_weight contracts over the tokens, of which there are many, into a result that
// may have fewer tiles than there are SMs. The tokens are then split, every split leaves
// its fp32 result in the workspace, and sum_splits_kernel adds them in order (the same
// result on every run). db is one more column of the product: dy^T times a column of ones,
// an MMA of 16 columns beside the tile's, so dy is read once for both.
#include "linear_few.cuh"
#include "product.cuh"

namespace swin {

namespace {

using prod::Matrix;
using prod::Params;
using prod::Tiling;

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapDataType kF32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;

Matrix rows_of(const void* p, int64_t rows, int64_t cols) { return Matrix{p, rows, cols, cols, rows * cols}; }

// out[i] = [old +] sum over the splits of part[s][i], i in fours; the last blocks do the same for
// the bias gradient. A block of 64 fours by kSumGroups threads each: a thread has all its splits'
// reads in flight and the groups are added in order. Bound by those reads' latency: the product
// has just left the partial results in L2.
constexpr int kSumGroups = 4, kSumWidth = 64;
template <typename T>
__global__ void __launch_bounds__(kSumGroups * kSumWidth)
    sum_splits_kernel(const float* __restrict__ part, int64_t n, int splits, T* __restrict__ out, bool add,
                      const float* __restrict__ bpart, int nb, float* __restrict__ bout) {
  __shared__ float4 group_sum[kSumGroups][kSumWidth];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % kSumWidth, grp = threadIdx.x / kSumWidth;
  const int64_t four = (int64_t)blockIdx.x * kSumWidth + lane, n4 = (n + 3) / 4;
  // the splits of this group
  const int s0 = splits * grp / kSumGroups, s1 = splits * (grp + 1) / kSumGroups;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int64_t j = four - n4;  // the bias gradient's element
  if (four < n4) {
#pragma unroll 8
    for (int s = s0; s < s1; ++s) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(part + (int64_t)s * n) + four);
      v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
    }
  } else if (bpart != nullptr && j < nb) {
#pragma unroll 8
    for (int s = s0; s < s1; ++s) v.x += __ldcg(bpart + (int64_t)s * nb + j);
  }
  group_sum[grp][lane] = v;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int k = 1; k < kSumGroups; ++k) {
    const float4 a = group_sum[k][lane];
    v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
  }
  if (four < n4) {
    if constexpr (sizeof(T) == 4) {
      float4* o = reinterpret_cast<float4*>(out) + four;
      if (add) v = make_float4(v.x + o->x, v.y + o->y, v.z + o->z, v.w + o->w);
      *o = v;
    } else {
      uint2* o = reinterpret_cast<uint2*>(out) + four;
      if (add) {
        const float2 a = prod::unpack_bf16(o->x), b = prod::unpack_bf16(o->y);
        v = make_float4(v.x + a.x, v.y + a.y, v.z + b.x, v.w + b.y);
      }
      *o = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    }
  } else if (bpart != nullptr && j < nb) {
    bout[j] = add ? bout[j] + v.x : v.x;
  }
}

// Few tokens, or few tiles of a long K, run as clusters (linear_few.cu), the rest as tiles: the
// one whose estimated time is shorter. A tile of fewer than 128 tokens brings its missing
// rows as zeros, more slowly than rows in memory (one token: 790 clocks a chunk; 128: 410).
// Measured, clusters against tiles: 1 token 6144x1536 8.4 and 40 us, 64 tokens 1536x6144 8.5 and
// 9.7 us, 100 tokens 192x768 8.4 and 4.5 us, 300 tokens 6144x1536 12.9 and 23.8 us, 500 tokens
// 1536x384 10.0 and 9.0 us.
constexpr int kFewTokens = 1024;
bool runs_as_clusters(const Tiling& t, const FewTiling& few, int64_t T, int64_t N, bool bmn) {
  if (T > kFewTokens) return false;
  double cost = prod::tiling_cost(t, T, N, 1, bmn, false);
  if (T < prod::kBM) cost += 0.9 * (1.0 - (double)T / prod::kBM) * t.chunks * prod::chunk_clocks(t.NT, t.cg, bmn);
  return few.cost < cost;
}

constexpr int kMaxSplits = 64;

Tiling weight_tiling(int64_t T, int K, int N) { return prod::choose_tiling(N, K, T, 1, true, kMaxSplits, true); }

}  // namespace

cudaError_t linear_launch(const void* x, const void* w, const float* b, const void* residual, void* y, void* pre,
                          int T, int K, int N, int act, int* status, cudaStream_t st) {
  const Tiling t = prod::choose_tiling(T, N, K, 1, false, 1, false);
  const FewTiling few = few_tiling(T, N, K);
  if (runs_as_clusters(t, few, T, N, false))
    return linear_few_launch(few, x, w, b, residual, y, pre, T, K, N, act, status, st);
  Params p{};
  p.M = T;
  p.N = N;
  p.act = act;
  p.bias = b;
  p.status = status;
  const Matrix r = rows_of(residual, T, N), z = rows_of(pre, T, N);
  prod::Extra ex;
  if (residual != nullptr) ex.aux = &r;
  if (pre != nullptr) ex.pre = &z;
  return prod::launch_product<false, false, prod::kEpiAct>(t, p, rows_of(x, T, K), rows_of(w, N, K), rows_of(y, T, N),
                                                           1, kBf16, kBf16, ex, st);
}

cudaError_t linear_bwd_data_launch(const void* dy, const void* w, const void* pre, void* dx, int T, int K, int N,
                                   int act, int* status, cudaStream_t st) {
  const Tiling t = prod::choose_tiling(T, K, N, 1, true, 1, false);
  const FewTiling few = few_tiling(T, K, N);
  if (runs_as_clusters(t, few, T, K, true))
    return linear_bwd_data_few_launch(few, dy, w, pre, dx, T, K, N, act, status, st);
  Params p{};
  p.M = T;
  p.N = K;
  p.act = act;
  p.status = status;
  const Matrix z = rows_of(pre, T, K);
  prod::Extra ex;
  if (act != SWIN_WATTN_ACT_NONE) ex.aux = &z;
  return prod::launch_product<false, true, prod::kEpiSlope>(t, p, rows_of(dy, T, N), rows_of(w, N, K),
                                                            rows_of(dx, T, K), 1, kBf16, kBf16, ex, st);
}

size_t linear_bwd_weight_workspace_bytes(int64_t T, int K, int N) {
  if (T == 0) return 256;
  const Tiling t = weight_tiling(T, K, N);
  return t.splits > 1 ? (size_t)t.splits * ((size_t)N * K + N) * 4 : 256;
}

// Launches of one linear_bwd_weight call.
int linear_bwd_weight_launches(int64_t T, int K, int N) { return T == 0 ? 0 : weight_tiling(T, K, N).splits > 1 ? 2 : 1; }

cudaError_t linear_bwd_weight_launch(const void* dy, const void* x, void* dw, float* db, int T, int K, int N,
                                     int dtype, int accumulate, void* workspace, int* status, cudaStream_t st) {
  const bool f32 = dtype == SWIN_WATTN_FP32;
  if (T == 0) {  // a sum over nothing
    if (accumulate) return cudaSuccess;
    cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)N * K * (f32 ? 4 : 2), st);
    if (e == cudaSuccess && db != nullptr) e = cudaMemsetAsync(db, 0, (size_t)N * 4, st);
    return e;
  }
  const Tiling t = weight_tiling(T, K, N);
  const Matrix a = rows_of(dy, T, N), b = rows_of(x, T, K);
  Params p{};
  p.M = N;
  p.N = K;
  p.status = status;
  p.k_sums = db;
  prod::Extra ex;
  if (t.splits == 1) {
    p.add_k_sums = accumulate != 0;
    const Matrix o = rows_of(dw, N, K);
    if (f32) {
      if (accumulate) p.old = static_cast<const float*>(dw);
      return prod::launch_product<true, true, prod::kEpiGrad32>(t, p, a, b, o, 1, kBf16, kF32, ex, st);
    }
    if (accumulate) ex.aux = &o;
    return prod::launch_product<true, true, prod::kEpiGrad16>(t, p, a, b, o, 1, kBf16, kBf16, ex, st);
  }
  float* part = static_cast<float*>(workspace);
  float* bpart = part + (size_t)t.splits * N * K;
  if (db != nullptr) p.k_sums = bpart;
  cudaError_t e = prod::launch_product<true, true, prod::kEpiGrad32>(t, p, a, b, rows_of(part, N, K), 1, kBf16, kF32,
                                                                     ex, st);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)N * K, fours = (n + 3) / 4 + (db != nullptr ? N : 0);
  const dim3 grid((unsigned)((fours + kSumWidth - 1) / kSumWidth)), block(kSumGroups * kSumWidth);
  if (f32)
    return launch_pdl(sum_splits_kernel<float>, grid, block, 0, st, (const float*)part, n, t.splits,
                      static_cast<float*>(dw), accumulate != 0, (const float*)(db != nullptr ? bpart : nullptr), N, db);
  return launch_pdl(sum_splits_kernel<__nv_bfloat16>, grid, block, 0, st, (const float*)part, n, t.splits,
                    static_cast<__nv_bfloat16*>(dw), accumulate != 0, (const float*)(db != nullptr ? bpart : nullptr),
                    N, db);
}

}  // namespace swin
