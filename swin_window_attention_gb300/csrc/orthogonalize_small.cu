// The Newton-Schulz update (orthogonalize.cu) of matrices whose smaller side is at most 128, in
// one launch. A cluster of CTAs keeps a matrix in shared memory for all its steps: each CTA a
// slab of the longer side (X in two fp16 parts, times 2^14), and all of A and B = a I + b A + c A^2.
// Per step
//   1. A's part from the slab on the tensor cores; the cluster's parts are summed in order
//      through distributed shared memory, each CTA adding up its share of the rows and handing
//      the rounded rows to the others;
//   2. A^2, and B from it;
//   3. the slab's two parts times B, written over the slab.
// Nothing but the matrix itself crosses memory, once in (twice, from L2, for its norm) and once
// out. What bounds it is latency: the steps' products depend on each other, and with the
// rounding, exchange and barriers between them take some 2 us each (96 x 384, five steps: 29.9 us;
// with X in one part 23.8 us). As separate launches of product.cuh's tiles they would take about
// 3.5 us each.
//
// The slab lies in blocks of 64 columns of 128-byte rows, 128-byte swizzled, so that one
// placement serves both products: for wide matrices (slab: all rows, a range of columns) the
// Gram product reads it K-major and the update MN-major, for tall ones (a range of rows, all
// columns) the other way round.
#include "product.cuh"
#include "orthogonalize.cuh"

namespace swin {

namespace {

using namespace prod;

constexpr int kSmThreads = 512, kSmWarps = kSmThreads / 32;
constexpr int kSide = 128;        // the smaller side at most
// Of the longer side, per CTA, at most: alone, or in a cluster, whose exchange of A's parts needs the
// room of two matrices.
constexpr int kSlabAlone = 384, kSlabShared = 256;
constexpr int kReadSide = 512;     // that the reads of G are laid out for
constexpr int kSmCluster = 8;
constexpr int kMatBytes = kSide * kSide * 2;
constexpr uint32_t kF16Format = (1u << 7) | (1u << 10);  // bits that make an operand bf16

struct SmallParams {
  const void* g;
  __nv_bfloat16* out;
  int rows, cols, steps, cluster, slab;  // slab: of the longer side, per CTA
  int slab_rows, slab_bytes;
  float eps, scale;
  int* status;
  uint64_t wait_ns;
  int fault;
};

__device__ __forceinline__ void store_cluster(uint32_t addr, uint2 v) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};\n" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
// One CTA has reached a point, with all its threads' accesses before it: an arrival on a barrier
// of another CTA, and the wait for all of them.
__device__ __forceinline__ void arrive_release_cluster(uint32_t mbar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(mbar) : "memory");
}
__device__ __forceinline__ bool wait_acquire_cluster(uint32_t mbar, uint32_t parity, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred q;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 q, [%1], %2;\n"
        " selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(ok)
        : "r"(mbar), "r"(parity)
        : "memory");
    if (ok) return true;
    uint64_t t1;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
    if (t0 == 0) t0 = t1;
    if (t1 - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ float load_cluster1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The value at an address, or 0 without a read where `in` is false: a predicated load, so that
// many are in flight (behind branches they came one after the other).
__device__ __forceinline__ float load_if(const float* a, bool in) {
  float v;
  asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %2, 0;\n mov.f32 %0, 0f00000000;\n @q ld.global.f32 %0, [%1];\n}\n"
               : "=f"(v)
               : "l"(a), "r"((uint32_t)in));
  return v;
}
__device__ __forceinline__ float load_if(const __nv_bfloat16* a, bool in) {
  uint16_t v;
  asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %2, 0;\n mov.u16 %0, 0;\n @q ld.global.u16 %0, [%1];\n}\n"
               : "=h"(v)
               : "l"(a), "r"((uint32_t)in));
  return __uint_as_float((uint32_t)v << 16);
}

// VEC: every row of G starts on a 16-byte boundary and holds a multiple of eight values, which are
// read eight at a time.
template <bool TALL, bool VEC, typename T>
__global__ void __launch_bounds__(kSmThreads, 1) orthogonalize_small_kernel(const SmallParams p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t s_tmem;
  __shared__ __align__(8) uint64_t s_bar[6];
  __shared__ float s_plain[kSmWarps];
  __shared__ Squares s_part[kSmWarps], s_norm;
  __shared__ __align__(16) float s_gain[kSide];  // the update's factors, a row or column of X each
  pdl_launch_dependents();
  const uint32_t smem0 = smem_u32(smem), bar = smem_u32(s_bar);  // A and A^2; the update's two halves; the cluster's exchanges
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int S = p.cluster, rank = blockIdx.x % S, mat = blockIdx.x / S;
  const int m = TALL ? p.cols : p.rows, n = TALL ? p.rows : p.cols;
  const int first = rank * p.slab, len = min(p.slab, n - first);  // this CTA's part of the longer side
  const int mp = (m + 15) & ~15;
  int bad = (smem0 & 1023u) != 0;

  // the slab's larger parts at 0, the smaller ones, A and B behind them. Alone, B is written over A:
  // each thread over the entries that it makes it from.
  unsigned char* sLow = smem + p.slab_bytes;
  unsigned char* sA = sLow + p.slab_bytes;
  const int b_off = S > 1 ? kMatBytes : 0;
  unsigned char* sB = sA + b_off;
  const uint32_t slab0 = smem0, low0 = slab0 + p.slab_bytes, a0 = low0 + p.slab_bytes, b0 = a0 + b_off;
  const int block = p.slab_rows * 128;  // bytes of 64 columns of the slab
  // element (r, c) of the slab; of A or B (blocks of 128 rows)
  auto at = [&](int r, int c) { return (c >> 6) * block + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) + (c & 7) * 2; };
  auto mat_at = [](int r, int c) { return (c >> 6) * (kSide * 128) + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) + (c & 7) * 2; };

  if (warp == 0) tc::tmem_alloc<512>(smem_u32(&s_tmem));
  if (tid == 0) {
    for (int i = 0; i < 6; ++i) tc::mbar_init(bar + 8 * i, i < 3 ? 1 : S);
    tc::mbar_init_fence();
  }
  for (int i = tid; i < p.slab_bytes / 8; i += kSmThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  pdl_wait();

  // ---- the slab of G: its share of the norm, then X = G / (|G| + eps) --------------------
  const int srows = TALL ? len : m, scols = TALL ? m : len;  // of the slab that hold G
  const int64_t origin = (int64_t)mat * p.rows * p.cols + (TALL ? (int64_t)first * p.cols : first);
  const T* g = static_cast<const T*>(p.g) + origin;
  const int c8 = scols / 8, n8 = srows * c8;  // VEC: scols is a multiple of 8
  const int quad = warp & 3, part = warp >> 2;  // tensor-memory lanes; columns
  const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
  // G is read once: it waits for its norm in tensor memory, which is idle until the steps. 32
  // values a thread at a time, `batch` to their columns of tensor memory:
  // with VEC, pieces of eight columns tid, tid + 512, ..., whose rows and columns advance by these;
  const int r_first = VEC ? tid / c8 : 0, c_first = tid - r_first * c8;
  const int r_step = VEC ? kSmThreads / c8 : 0, c_step = kSmThreads - r_step * c8;
  auto advance = [&](int& r, int& c) {
    r += r_step;
    c += c_step;
    if (c >= c8) {
      c -= c8;
      ++r;
    }
  };
  // else kRows rows (16 apart) of kGroups groups of 32 columns, a lane each. (Element by element
  // as the pieces, the addresses alone took 12 us of one 97 x 385.)
  constexpr int kGroups = TALL ? kSide / 32 : kReadSide / 32, kRows = 32 / kGroups;
  constexpr int kBatches = kSide * kReadSide / 32 / kSmThreads;
  // place in the slab's row r of the lane's column of group j
  auto at_group = [&](int r, int j) {
    return (j >> 1) * block + r * 128 + (((lane >> 3) + 4 * (j & 1) ^ (r & 7)) << 4) + (lane & 7) * 2;
  };
  auto batch_begins = [&](int batch) {
    return VEC ? (tid & ~31) + 4 * batch * kSmThreads < n8 : warp + kSmWarps * kRows * batch < srows;
  };
  Squares total;
  {
    float2 plain = make_float2(0.0f, 0.0f);
    int r = r_first, c = c_first;
#pragma unroll 1
    for (int batch = 0; batch < kBatches; ++batch) {
      if (!batch_begins(batch)) break;
      float v[4][8];
      if constexpr (VEC) {
        const int i = 4 * batch * kSmThreads + tid;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (i + u * kSmThreads < n8) {
            load8(g + (int64_t)r * p.cols + c * 8, v[u]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
          }
          advance(r, c);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          const int row = warp + kSmWarps * (batch * kRows + u / kGroups), col = lane + u % kGroups * 32;
          v[u >> 3][u & 7] = load_if(g + (int64_t)row * p.cols + col, row < srows && col < scols);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) add_plain(v[u], plain);
      uint32_t w[32];
#pragma unroll
      for (int u = 0; u < 32; ++u) w[u] = __float_as_uint(v[u >> 3][u & 7]);
      __syncwarp();
      tc::st_x32(trow + part * 128 + batch * 32, w);
    }
    tc::wait_st();
    const float w = warp_sum(plain.x + plain.y);
    if (lane == 0) s_plain[warp] = w;
    __syncthreads();
    total = {s_plain[0], 0.0f, 0.0f};
#pragma unroll
    for (int w = 1; w < kSmWarps; ++w) total.mid += s_plain[w];
    if (!plain_sum_holds(total.mid)) {
      Squares sum{};
      for (int r = warp; r < srows; r += kSmWarps)
        for (int c = lane; c < scols; c += 32) add_square(load_f32(g + (int64_t)r * p.cols + c), sum);
      sum = warp_sum(sum);
      if (lane == 0) s_part[warp] = sum;
      __syncthreads();
      total = s_part[0];
      for (int w = 1; w < kSmWarps; ++w) add(total, s_part[w]);
    }
  }
  if (S > 1) {
    if (tid == 0) s_norm = total;
    cluster_sync_all();
    total = {};
    for (int s = 0; s < S; ++s) {
      const uint32_t peer = map_to_rank(smem_u32(&s_norm), s);
      add(total, {load_cluster1(peer), load_cluster1(peer + 4), load_cluster1(peer + 8)});
    }
  }
  const Inverse k = inverse_of(total, p.eps);
  {
    int r = r_first, c = c_first;
#pragma unroll 1
    for (int batch = 0; batch < kBatches; ++batch) {
      if (!batch_begins(batch)) break;
      uint32_t w[32];
      tc::ld32_wait(trow + part * 128 + batch * 32, w);
      float v[32];
#pragma unroll
      for (int u = 0; u < 32; ++u) v[u] = __uint_as_float(w[u]) * k.pre * k.inv;
      if constexpr (VEC) {
        const int i = 4 * batch * kSmThreads + tid;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t o[4], l[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) two_parts(make_float2(v[8 * u + 2 * e], v[8 * u + 2 * e + 1]), o[e], l[e]);
          if (i + u * kSmThreads < n8) {
            const int to = at(r, 8 * c);
            *reinterpret_cast<uint4*>(smem + to) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(sLow + to) = make_uint4(l[0], l[1], l[2], l[3]);
          }
          advance(r, c);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          const int row = warp + kSmWarps * (batch * kRows + u / kGroups), col = lane + u % kGroups * 32;
          if (row < srows && col < scols) {
            const int to = at_group(row, u % kGroups);
            const __half h = __float2half_rn(v[u]);
            *reinterpret_cast<__half*>(smem + to) = h;
            *reinterpret_cast<__half*>(sLow + to) = __float2half_rn(v[u] - __half2float(h));
          }
        }
      }
    }
  }
  tc::fence_proxy_async();
  tc::fence_before_sync();
  __syncthreads();

  // ---- the steps ------------------------------------------------------------------------
  constexpr uint32_t kHi = desc_hi(1024, kSW128);
  const uint32_t id_gram = (tc::idesc_bf16(kSide, 16, TALL, TALL) ^ kF16Format) + ((uint32_t)(mp - 16) >> 3 << 17);
  const uint32_t id_mat = (tc::idesc_bf16(kSide, 16, false, false) ^ kF16Format) + ((uint32_t)(mp - 16) >> 3 << 17);
  // Warp 0 issues; every thread waits for the products to complete.
  auto issue = [&](auto mmas) {
    if (warp == 0 && !bad) {
      tc::fence_after_sync();
      if (elect_one()) mmas();
      __syncwarp();
    }
  };
  auto commit_products = [&](int i) {
#ifdef SWIN_WATTN_FAULT_INJECTION
    if (p.fault != kFaultGemm)
#endif
      tc::commit(bar + 8 * i);
  };
  auto wait_products = [&](int i, uint32_t parity) {
    if (!bad && !warp_wait(bar + 8 * i, parity, p.wait_ns)) bad = 1;
    tc::fence_after_sync();
  };
  // Every CTA of the cluster has reached exchange i of this step: one thread a peer releases for
  // its CTA. (As fast as a cluster barrier, but a product that never completes in one CTA ends
  // in this wait's limit, and the status says so.)
  auto exchange = [&](int i, uint32_t parity) {
    __syncthreads();
    if (tid < S) arrive_release_cluster(map_to_rank(bar + 8 * (3 + i), tid));
    if (!bad && !__all_sync(0xffffffffu, wait_acquire_cluster(bar + 8 * (3 + i), parity, p.wait_ns))) bad = 1;
  };
  const int row = quad * 32 + lane;
  const int k_steps = (len + 15) / 16;  // of the Gram product
  const int m_steps = mp / 16;
  const uint32_t block_d = block >> 4;  // in a descriptor's units
  // A's part, the K steps [t0, t1): columns [0, mp) of the accumulator
  auto gram = [&](int t0, int t1) {
    uint32_t x = TALL ? desc_lo(slab0, block) + t0 * 128 : desc_lo(slab0, 16) + (t0 >> 2) * block_d + (t0 & 3) * 2;
    for (int t = t0; t < t1; ++t) {
      mma<1>(tmem, x, kHi, x, kHi, id_gram, t > 0);
      x += TALL ? 128 : (t & 3) == 3 ? block_d - 6 : 2;
    }
  };
  uint32_t phase = 0;
  issue([&]() {
    gram(0, k_steps);
    commit_products(0);
  });

  float mu = first_shift(m);
  for (int step = 0; step < p.steps; ++step) {
    const bool last = step == p.steps - 1;
    const float alpha = last ? p.scale / (kScale * kScaleX) : 1.0f / kScale;
    constexpr float kToA = kScale / (kScaleX * kScaleX);  // (2^14 X)(2^14 X)^T = 2^28 A -> 2^8 A
    const NsStep ns = ns_step(mu);
    mu = next_shift(mu);
    wait_products(0, phase);
    phase ^= 1;
    const int c0 = part * 32;
    if (S == 1) {
      if (c0 < mp) {
        uint32_t a[32];
        tc::ld32_wait(trow + c0, a);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            o[q] = pack_f16(__uint_as_float(a[8 * c + 2 * q]) * kToA, __uint_as_float(a[8 * c + 2 * q + 1]) * kToA);
          *reinterpret_cast<uint4*>(sA + mat_at(row, c0 + 8 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (part == quad)
          *reinterpret_cast<__half*>(sA + mat_at(row, row)) = __float2half_rn(fmaf(of_lane(a, lane), kToA, -ns.mu * kScale));
      }
    } else {
      // fp32 parts [128][128] over A and B, of which nothing is needed any more; 16-byte pieces
      // of a row swizzled against bank conflicts
      float* fp = reinterpret_cast<float*>(sA);
      auto f_at = [](int r, int c4) { return r * kSide + ((c4 ^ (r & 7)) << 2); };  // c4: piece of four columns
      if (c0 < mp) {
        uint32_t a[32];
        tc::ld32_wait(trow + c0, a);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(fp + f_at(row, c0 / 4 + c)) = make_uint4(a[4 * c], a[4 * c + 1], a[4 * c + 2], a[4 * c + 3]);
      }
      tc::fence_before_sync();
      exchange(0, step & 1);
      // Rows rank, rank + S, ...: a thread sums four columns of a row over the cluster, a warp
      // whole rows, so that what it reads of another CTA at once is contiguous (2048 x 128, read
      // by scattered pieces it took 16 us more).
      constexpr int kMine = kSide / 2 * (kSide / 4) / kSmThreads;  // at S = 2, pieces per thread
      uint2 mine[kMine];
      const int my_rows = (mp - rank + S - 1) / S, pieces = mp / 4;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int e = tid + i * kSmThreads, r = rank + e / pieces * S, c = e % pieces;
        if (e < my_rows * pieces) {
          float4 u = make_float4(0, 0, 0, 0);
          for (int s = 0; s < S; ++s) {
            const float4 x = load_cluster4(map_to_rank(a0, s) + f_at(r, c) * 4);
            u = make_float4(u.x + x.x, u.y + x.y, u.z + x.z, u.w + x.w);
          }
          if (c == r >> 2) {
            const float v = -ns.mu * (kScaleX * kScaleX);
            u = make_float4(u.x + ((r & 3) == 0 ? v : 0.0f), u.y + ((r & 3) == 1 ? v : 0.0f),
                            u.z + ((r & 3) == 2 ? v : 0.0f), u.w + ((r & 3) == 3 ? v : 0.0f));
          }
          mine[i] = make_uint2(pack_f16(u.x * kToA, u.y * kToA), pack_f16(u.z * kToA, u.w * kToA));
        }
      }
      exchange(1, step & 1);  // every part has been read
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int e = tid + i * kSmThreads, r = rank + e / pieces * S, c = e % pieces;
        if (e < my_rows * pieces)
          for (int s = 0; s < S; ++s) store_cluster(map_to_rank(a0 + mat_at(r, 4 * c), s), mine[i]);
      }
      tc::fence_proxy_async();
      exchange(2, step & 1);  // A is complete in every CTA
    }
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();

    // A^2 behind the Gram accumulator, then B
    issue([&]() {
      uint32_t x = desc_lo(a0, 16);
      for (int t = 0; t < m_steps; ++t) {
        mma<1>(tmem + kSide, x, kHi, x, kHi, id_mat, t > 0);
        x += (t & 3) == 3 ? (kSide * 128 >> 4) - 6 : 2;
      }
      commit_products(0);
    });
    wait_products(0, phase);
    phase ^= 1;
    if (c0 < mp) {
      uint32_t a[32];
      tc::ld32_wait(trow + kSide + c0, a);
      const float x_diag = part == quad ? __half2float(*reinterpret_cast<const __half*>(sA + mat_at(row, row))) : 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(sA + mat_at(row, c0 + 8 * c));
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = 8 * c + 2 * q;
          const float2 x = unpack_f16(in[q]);
          o[q] = pack_f16(fmaf(__uint_as_float(a[e]), kNsC / kScale, x.x * ns.b),
                          fmaf(__uint_as_float(a[e + 1]), kNsC / kScale, x.y * ns.b));
        }
        *reinterpret_cast<uint4*>(sB + mat_at(row, c0 + 8 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (part == quad) {
        const float exact = fmaf(of_lane(a, lane), kNsC / kScale, fmaf(x_diag, ns.b, ns.e * kScale));
        const __half held = __float2half_rn(exact);
        *reinterpret_cast<__half*>(sB + mat_at(row, row)) = held;
        s_gain[row] = alpha * __fdividef(exact, __half2float(held));
      }
    }
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();

    // The slab times B, in two halves: wide, 128 rows by up to 256 columns each; tall, two tiles
    // of 128 rows by mp columns each.
    const int halves = TALL ? (p.slab_rows + 255) / 256 : (len + 255) / 256;
    issue([&]() {
      for (int h = 0; h < halves; ++h) {
        if constexpr (TALL) {
          for (int tile = 2 * h; tile < min(2 * h + 2, p.slab_rows / kSide); ++tile) {
            for (int high = 0; high < 2; ++high) {  // the smaller part first
              uint32_t x = desc_lo((high ? slab0 : low0) + tile * (kSide * 128), 16), y = desc_lo(b0, 16);
              for (int t = 0; t < m_steps; ++t) {
                mma<1>(tmem + tile * kSide, x, kHi, y, kHi, id_mat, t + high > 0);
                x += (t & 3) == 3 ? block_d - 6 : 2;
                y += (t & 3) == 3 ? (kSide * 128 >> 4) - 6 : 2;
              }
            }
          }
        } else {
          const int c = 256 * h, nn = min(256, (len - c + 15) & ~15);
          const uint32_t id = (tc::idesc_bf16(kSide, 16, true, false) ^ kF16Format) + ((uint32_t)(nn - 16) >> 3 << 17);
          for (int high = 0; high < 2; ++high) {  // the smaller part first
            uint32_t x = desc_lo(b0, 16), y = desc_lo((high ? slab0 : low0) + 4 * h * block, block);
            for (int t = 0; t < m_steps; ++t) {
              mma<1>(tmem + c, x, kHi, y, kHi, id, t + high > 0);
              x += (t & 3) == 3 ? (kSide * 128 >> 4) - 6 : 2;
              y += 128;
            }
          }
        }
        commit_products(1 + h);
      }
    });
    // The accumulator's 32-column pieces, four quadrants' rows each: wide, piece = columns; tall,
    // tile of 128 rows and columns. After each round of four pieces the next step's Gram product
    // takes the 128 columns (rows) that are complete; its accumulator is the first piece's place,
    // which has been read by then.
    const int tiles32 = (mp + 31) / 32;
    const int n_pieces = TALL ? p.slab_rows / kSide * tiles32 : (len + 31) / 32;
    int waited = 0, begun = 0;  // halves; K steps
    for (int i0 = 0; i0 < n_pieces; i0 += 4) {
      const int i = i0 + part, i_last = min(i0 + 3, n_pieces - 1);
      // every thread waits for the halves that hold the round's pieces
      const int need = (TALL ? i_last / tiles32 / 2 : i_last / 8) + 1;
      for (; waited < need; ++waited) wait_products(1 + waited, step & 1);
      if (i < n_pieces) {
        const int r = TALL ? i / tiles32 * kSide + row : row, c = (TALL ? i % tiles32 : i) * 32;
        const uint32_t col = TALL ? (uint32_t)(i / tiles32 * kSide + c) : (uint32_t)c;
        uint32_t a[32];
        tc::ld32_wait(trow + col, a);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t o[4], l[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 f = TALL ? *reinterpret_cast<const float2*>(&s_gain[c + 8 * k + 2 * q]) : splat(s_gain[row]);
            const float2 x = __fmul2_rn(make_float2(__uint_as_float(a[8 * k + 2 * q]), __uint_as_float(a[8 * k + 2 * q + 1])), f);
            if (last)
              o[q] = pack_bf16(x.x, x.y);
            else
              two_parts(x, o[q], l[q]);
          }
          const int to = at(r, c + 8 * k);
          *reinterpret_cast<uint4*>(smem + to) = make_uint4(o[0], o[1], o[2], o[3]);
          if (!last) *reinterpret_cast<uint4*>(sLow + to) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
      tc::fence_proxy_async();
      tc::fence_before_sync();
      __syncthreads();
      if (!last) {
        const bool end = i0 + 4 >= n_pieces;
        const int complete = end ? k_steps : min(k_steps, 8 * (TALL ? (i0 + 4) / tiles32 : i0 / 4 + 1));
        issue([&]() {
          gram(begun, complete);
          if (end) commit_products(0);
        });
        begun = complete;
      }
    }
  }

  // ---- the result, from the slab in bf16 -------------------------------------------------
  __nv_bfloat16* out = p.out + origin;
  if (p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0) {
    for (int i = tid; i < n8; i += kSmThreads) {
      const int r = i / c8, c = i % c8 * 8;
      *reinterpret_cast<uint4*>(out + (int64_t)r * p.cols + c) = *reinterpret_cast<const uint4*>(smem + at(r, c));
    }
  } else {
    for (int r = warp; r < srows; r += kSmWarps) {
      __nv_bfloat16 v[kGroups];
#pragma unroll
      for (int j = 0; j < kGroups; ++j)
        if (lane + j * 32 < scols) v[j] = *reinterpret_cast<const __nv_bfloat16*>(smem + at_group(r, j));
#pragma unroll
      for (int j = 0; j < kGroups; ++j)
        if (lane + j * 32 < scols) out[(int64_t)r * p.cols + lane + j * 32] = v[j];
    }
  }
  if (bad && p.status != nullptr) atomicOr(p.status, 1);
  // no CTA leaves while another may still read its parts
  if (S > 1) cluster_sync_all();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc<512>(tmem);
}

template <bool TALL, typename T>
cudaError_t launch_small(SmallParams p, int count, cudaStream_t st) {
  const int n = TALL ? p.rows : p.cols;
  // One CTA where the matrix fits it (no exchange); else the largest cluster that leaves every
  // matrix of the stack resident at once (128 x 512: in clusters of eight 41 us, of two 46 us;
  // sixteen 100 x 1500: of six 60 us, of eight in two rounds 105 us). Slabs are multiples of 64,
  // none empty.
  p.cluster = n <= kSlabAlone ? 1 : (n + kSlabShared - 1) / kSlabShared;
  if (p.cluster > 1)
    for (int s = p.cluster + 1; s <= kSmCluster; ++s)
      if (count <= kResidentClusters[s]) p.cluster = s;
  p.slab = ((n + p.cluster - 1) / p.cluster + 63) / 64 * 64;
  p.cluster = (n + p.slab - 1) / p.slab;
  p.slab_rows = TALL ? (p.slab + kSide - 1) / kSide * kSide : kSide;
  p.slab_bytes = TALL ? 2 * p.slab_rows * 128 : p.slab / 64 * (kSide * 128);
  p.wait_ns = wait_limit_ns();
  p.fault = fault_site();
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const int smem = std::max(120 * 1024, 2 * p.slab_bytes + (p.cluster > 1 ? 2 : 1) * kMatBytes);
  const bool vec = p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(p.g) % 16 == 0;
  auto kern = vec ? orthogonalize_small_kernel<TALL, true, T> : orthogonalize_small_kernel<TALL, false, T>;
  static std::atomic<uint64_t> allowed[2];
  e = allow_smem(reinterpret_cast<const void*>(kern), di.smem_max - 1024, di.device, &allowed[vec]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(count * p.cluster));
  cfg.blockDim = dim3(kSmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

bool orthogonalize_small_applies(int rows, int cols) {
  return std::min(rows, cols) <= kSide && std::max(rows, cols) <= kSlabShared * kSmCluster;
}

cudaError_t orthogonalize_small_launch(const void* g, void* out, int count, int rows, int cols, int dtype, int steps,
                                       float eps, float scale, int* status, cudaStream_t st) {
  SmallParams p{};
  p.g = g;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.rows = rows;
  p.cols = cols;
  p.steps = steps;
  p.eps = eps;
  p.scale = scale;
  p.status = status;
  const bool f32 = dtype == SWIN_WATTN_FP32;
  if (rows > cols) return f32 ? launch_small<true, float>(p, count, st) : launch_small<true, __nv_bfloat16>(p, count, st);
  return f32 ? launch_small<false, float>(p, count, st) : launch_small<false, __nv_bfloat16>(p, count, st);
}

}  // namespace swin
