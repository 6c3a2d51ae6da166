// The norm over all gradients of a model, and their clipping:
//   n = scale |g|,   out = g * scale * min(1, max_norm / (n + eps))
// over any number of fp32 and bf16 tensors of any size and alignment. The tensors are cut into
// pieces, which blocks take in turn, so that one launch covers hundreds of tensors of all sizes;
// their addresses and lengths travel as kernel parameters, a table of up to 1024 tensors a launch.
// * squares_kernel: a block's sum of squares in 64 bits, one for each block, in the workspace.
// * scale_kernel: every block adds those up in the same order (the same bits on every run),
//   forms the factor, and scales its pieces, from the last one back: what the first launch read
//   last is still in L2.
// Where the factor is 1 and the tensors are scaled in place there is nothing to write.
#include <algorithm>
#include <new>

#include "common.cuh"

namespace swin {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 4 * 152;

template <int N>
struct Table {
  const void* in[N];
  void* out[N];
  int64_t n_bf16[N];  // 2 * elements + (1 for bf16)
  uint32_t first[N];  // the number of pieces before this tensor's
  int count;
  uint32_t pieces, piece;  // all pieces; elements of one
};

struct Piece {
  const void* in;
  void* out;
  int64_t begin;
  int len;
  bool bf16;
};

// Piece number i: the last tensor whose first piece is at most i.
template <int N>
__device__ __forceinline__ Piece piece_of(const Table<N>& t, uint32_t i) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  Piece p;
  const int64_t n = t.n_bf16[lo] >> 1;
  p.bf16 = t.n_bf16[lo] & 1;
  p.in = t.in[lo];
  p.out = t.out[lo];
  p.begin = (int64_t)(i - t.first[lo]) * t.piece;
  p.len = (int)min((int64_t)t.piece, n - p.begin);
  return p;
}

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// 16 bytes as fp32 values.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[16 / sizeof(T)]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(in[i]);
    } else {
      v[2 * i] = __uint_as_float(in[i] << 16);
      v[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
    }
  }
}

// Elements before the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int len) {
  return min(len, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T));
}

constexpr int kLoads = 4;  // 16-byte loads of a thread in flight

// The squares of up to 64 bytes a thread are summed in fp32 and joined to the block's sum in 64 bits.
// That holds where the fp32 sum comes out between these bounds: no square has overflowed, and those
// lost are nothing beside it. Else (tiny, huge or no values, NaN) they are summed again in 64 bits.
__device__ __forceinline__ bool holds(float s) { return s >= 0x1p-60f && s <= 0x1p96f; }

template <typename T>
__device__ double squares(const T* p, int len) {
  constexpr int kPer = 16 / sizeof(T);
  const int head = head_of(p, len), vecs = (len - head) / kPer, tail = head + vecs * kPer;
  double sum = 0.0;
  if ((int)threadIdx.x < head) {
    const double v = value(p + threadIdx.x);
    sum += v * v;
  }
  if (tail + (int)threadIdx.x < len) {
    const double v = value(p + tail + threadIdx.x);
    sum += v * v;
  }
  const uint4* body = reinterpret_cast<const uint4*>(p + head);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kThreads * kLoads) {
    uint4 w[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) w[k] = i0 + k * kThreads < vecs ? body[i0 + k * kThreads] : make_uint4(0, 0, 0, 0);
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      float v[kPer];
      unpack<T>(w[k], v);
#pragma unroll
      for (int e = 0; e < kPer; e += 2) s = __ffma2_rn(make_float2(v[e], v[e + 1]), make_float2(v[e], v[e + 1]), s);
    }
    const float all = s.x + s.y;
    if (holds(all)) {
      sum += (double)all;
    } else {
      uint32_t bits = 0;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) bits |= w[k].x | w[k].y | w[k].z | w[k].w;
      if ((bits & 0x7fff7fffu) == 0) continue;  // zeros
#pragma unroll 1
      for (int k = 0; k < kLoads; ++k) {
        float v[kPer];
        unpack<T>(w[k], v);
#pragma unroll
        for (int e = 0; e < kPer; ++e) sum = fma((double)v[e], (double)v[e], sum);
      }
    }
  }
  return sum;
}

// The sum over the block, in every thread.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double warps[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += warps[w];
  return v;
}

template <int N>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<N> t, double* partial) {
  pdl_launch_dependents();
  pdl_wait();
  double sum = 0.0;
  for (uint32_t i = blockIdx.x; i < t.pieces; i += gridDim.x) {
    const Piece p = piece_of(t, i);
    sum += p.bf16 ? squares(static_cast<const __nv_bfloat16*>(p.in) + p.begin, p.len)
                  : squares(static_cast<const float*>(p.in) + p.begin, p.len);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void scale_one(const T* in, T* out, float factor) {
  const float v = value(in) * factor;
  if constexpr (sizeof(T) == 4)
    *out = v;
  else
    *out = __float2bfloat16_rn(v);
}

template <typename T>
__device__ void scale_piece(const T* in, T* out, int len, float factor) {
  constexpr int kPer = 16 / sizeof(T);
  if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
    for (int i = threadIdx.x; i < len; i += kThreads) scale_one(in + i, out + i, factor);
    return;
  }
  const int head = head_of(in, len), vecs = (len - head) / kPer, tail = head + vecs * kPer;
  if ((int)threadIdx.x < head) scale_one(in + threadIdx.x, out + threadIdx.x, factor);
  if (tail + (int)threadIdx.x < len) scale_one(in + tail + threadIdx.x, out + tail + threadIdx.x, factor);
  const uint4* from = reinterpret_cast<const uint4*>(in + head);
  uint4* to = reinterpret_cast<uint4*>(out + head);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kThreads * kLoads) {
    uint4 w[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (i0 + k * kThreads < vecs) w[k] = from[i0 + k * kThreads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      if (i0 + k * kThreads >= vecs) break;
      float v[kPer];
      unpack<T>(w[k], v);
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] *= factor;
      uint4 o;
      if constexpr (sizeof(T) == 4)
        o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      else
        o = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      to[i0 + k * kThreads] = o;
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(const __grid_constant__ Table<N> t, const double* partial, int n_partial, float max_norm, float scale,
                 float eps, bool in_place, float* norm) {
  pdl_launch_dependents();
  pdl_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < n_partial; i += kThreads) sum += __ldcg(partial + i);
  const float n = (float)((double)scale * sqrt(block_sum(sum)));
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float c = __fdiv_rn(max_norm, n + eps);
  const float factor = scale * (c > 1.0f ? 1.0f : c);  // NaN stays NaN
  if (in_place && factor == 1.0f) return;
  for (uint32_t i = blockIdx.x; i < t.pieces; i += gridDim.x) {
    const Piece p = piece_of(t, t.pieces - 1 - i);
    if (p.bf16)
      scale_piece(static_cast<const __nv_bfloat16*>(p.in) + p.begin, static_cast<__nv_bfloat16*>(p.out) + p.begin, p.len, factor);
    else
      scale_piece(static_cast<const float*>(p.in) + p.begin, static_cast<float*>(p.out) + p.begin, p.len, factor);
  }
}

// Elements of a piece: some four pieces for each block that fits, of 2048 to 16384 elements (a thread's
// loads are then 16 bytes times kLoads and a few times that).
uint32_t piece_of_total(int64_t total) {
  int64_t piece = 2048;
  while (piece < 16384 && total / piece > 4 * kMaxBlocks) piece *= 2;
  return (uint32_t)piece;
}

constexpr int kFewEntries = 64, kManyEntries = 1024;

template <int N>
cudaError_t run(const Table<N>* tables, int n_tables, bool in_place, float max_norm, float scale, float eps, float* norm,
                double* partial, cudaStream_t st) {
  int n_partial = 0;
  for (int i = 0; i < n_tables; ++i) {
    const int blocks = (int)std::min<uint32_t>(tables[i].pieces, kMaxBlocks);
    if (blocks == 0) continue;  // no elements at all: the norm is zero
    const cudaError_t e = launch_pdl(squares_kernel<N>, dim3(blocks), dim3(kThreads), 0, st, tables[i], partial + n_partial);
    if (e != cudaSuccess) return e;
    n_partial += blocks;
  }
  for (int i = 0; i < n_tables; ++i) {
    const int blocks = std::max(1, (int)std::min<uint32_t>(tables[i].pieces, kMaxBlocks));
    const cudaError_t e = launch_pdl(scale_kernel<N>, dim3(blocks), dim3(kThreads), 0, st, tables[i], (const double*)partial,
                                     n_partial, max_norm, scale, eps, in_place, i == 0 ? norm : (float*)nullptr);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N>
Table<N>* make_tables(const void* const* in, void* const* out, const int64_t* sizes, const int* dtypes, int count,
                      int n_tables, uint32_t piece) {
  Table<N>* t = new (std::nothrow) Table<N>[n_tables]();
  if (t == nullptr) return nullptr;
  int k = 0;
  for (int i = 0; i < n_tables; ++i) t[i].piece = piece;
  for (int i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    if (t[k].count == N) ++k;
    Table<N>& to = t[k];
    to.in[to.count] = in[i];
    to.out[to.count] = out[i];
    to.n_bf16[to.count] = sizes[i] * 2 + (dtypes[i] == SWIN_WATTN_BF16 ? 1 : 0);
    to.first[to.count++] = to.pieces;
    to.pieces += (uint32_t)((sizes[i] + piece - 1) / piece);
  }
  return t;
}

}  // namespace

// A plan's tables. `few` or `many` by the number of tensors that have elements.
struct ClipTables {
  int n_tables;
  bool in_place;
  Table<kFewEntries>* few;
  Table<kManyEntries>* many;
};

ClipTables* clip_tables_make(const void* const* in, void* const* out, const int64_t* sizes, const int* dtypes, int count) {
  int64_t total = 0;
  int used = 0;
  bool in_place = true;
  for (int i = 0; i < count; ++i) {
    total += sizes[i];
    used += sizes[i] > 0;
    in_place = in_place && (sizes[i] == 0 || in[i] == out[i]);
  }
  ClipTables* c = new (std::nothrow) ClipTables{};
  if (c == nullptr) return nullptr;
  const uint32_t piece = piece_of_total(total);
  const int per = used <= kFewEntries ? kFewEntries : kManyEntries;
  c->n_tables = std::max(1, (used + per - 1) / per);
  c->in_place = in_place;
  if (per == kFewEntries)
    c->few = make_tables<kFewEntries>(in, out, sizes, dtypes, count, c->n_tables, piece);
  else
    c->many = make_tables<kManyEntries>(in, out, sizes, dtypes, count, c->n_tables, piece);
  if (c->few == nullptr && c->many == nullptr) {
    delete c;
    return nullptr;
  }
  return c;
}
void clip_tables_free(ClipTables* c) {
  if (c == nullptr) return;
  delete[] c->few;
  delete[] c->many;
  delete c;
}
size_t clip_workspace_bytes(const ClipTables* c) { return (size_t)c->n_tables * kMaxBlocks * sizeof(double); }
int clip_launches(const ClipTables* c) {
  const uint32_t pieces = c->few != nullptr ? c->few->pieces : c->many->pieces;  // only a single table can be empty
  return c->n_tables * 2 - (pieces == 0 ? 1 : 0);
}
cudaError_t clip_launch(const ClipTables* c, float max_norm, float scale, float eps, float* norm, void* workspace,
                        cudaStream_t st) {
  double* partial = static_cast<double*>(workspace);
  return c->few != nullptr ? run(c->few, c->n_tables, c->in_place, max_norm, scale, eps, norm, partial, st)
                           : run(c->many, c->n_tables, c->in_place, max_norm, scale, eps, norm, partial, st);
}

}  // namespace swin
