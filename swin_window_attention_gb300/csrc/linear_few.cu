// linear and linear_bwd_data for few tokens, or few tiles of a long K: the product is then bound by
// reading the weight, and by latency. Against the tiles of product.cuh:
// * the weight's rows are the MMA's 128 rows and the tokens its N (16 to 128), so no row of
//   a tile is padding: the result arrives transposed, a thread holding one output channel of
//   every token, and is stored 64 bytes per warp and token;
// * a cluster of up to eight CTAs shares a tile, each over its part of K, so that some 150
//   CTAs read the weight whatever its shape. Their partial results are summed in order
//   through distributed shared memory, each CTA finishing its share of the tokens.
#include "linear_few.cuh"
#include "product.cuh"

namespace swin {

namespace {

using namespace prod;

constexpr int kFewTmem = 128;  // columns: the accumulator
constexpr int kFewEpi = 16, kFewMMA = kFewEpi, kFewCOPY = kFewEpi + 1, kFewWarps = kFewEpi + 2;
constexpr int kMaxCluster = 8, kMaxTN = 128;
constexpr int kFullBar = 0, kEmptyBar = kMaxStages, kDoneBar = 2 * kMaxStages, kFewBars = kDoneBar + 1;

struct FewParams {
  int T, N, TN;     // tokens, result columns, tokens per tile (the MMA's N)
  int n_tiles;      // tiles along N
  int chunks;       // of K
  int cluster;      // CTAs per tile
  int stages, stage_bytes;
  int off_bar;
  uint32_t idesc;
  int act;
  const float* bias;
  const __nv_bfloat16* aux;  // residual, or pre-activation
  __nv_bfloat16* out;
  __nv_bfloat16* pre;
  int* status;
  uint64_t wait_ns;
  int fault;
};

__device__ __forceinline__ float load_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float bf16_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <int EPI>
__device__ __forceinline__ float finish(float acc, float bias, float aux, int act, float* z) {
  if constexpr (EPI == kEpiAct) {
    const float2 v = make_float2(acc + bias, 0.0f);
    *z = v.x;
    float y = v.x;
    switch (act) {
      case SWIN_WATTN_ACT_RELU: y = act_value<SWIN_WATTN_ACT_RELU>(v).x; break;
      case SWIN_WATTN_ACT_GELU: y = act_value<SWIN_WATTN_ACT_GELU>(v).x; break;
      case SWIN_WATTN_ACT_GELU_TANH: y = act_value<SWIN_WATTN_ACT_GELU_TANH>(v).x; break;
      case SWIN_WATTN_ACT_SILU: y = act_value<SWIN_WATTN_ACT_SILU>(v).x; break;
    }
    return y + aux;
  } else {
    const float2 v = make_float2(aux, 0.0f);
    switch (act) {
      case SWIN_WATTN_ACT_RELU: return acc * act_slope<SWIN_WATTN_ACT_RELU>(v).x;
      case SWIN_WATTN_ACT_GELU: return acc * act_slope<SWIN_WATTN_ACT_GELU>(v).x;
      case SWIN_WATTN_ACT_GELU_TANH: return acc * act_slope<SWIN_WATTN_ACT_GELU_TANH>(v).x;
      case SWIN_WATTN_ACT_SILU: return acc * act_slope<SWIN_WATTN_ACT_SILU>(v).x;
    }
    return acc;
  }
}

// WMN: the weight is read MN-major (its rows are K of the product: dy W).
template <bool WMN, int EPI>
__global__ void __launch_bounds__(kFewWarps * 32, 1)
    few_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map, const FewParams p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  pdl_launch_dependents();
  const uint32_t smem0 = smem_u32(smem), bar0 = smem0 + p.off_bar;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // cluster -> 128 output channels from n0 of the TN tokens from t00
  const int S = p.cluster, rank = blockIdx.x % S, tile = blockIdx.x / S;
  const int n0 = tile % p.n_tiles * kBM, t00 = tile / p.n_tiles * p.TN, tokens = min(p.TN, p.T - t00);
  // this CTA's chunks of K
  const int c0 = (int)((int64_t)p.chunks * rank / S), c1 = (int)((int64_t)p.chunks * (rank + 1) / S);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + p.off_bar + 8 * kFewBars);
  int bad = (smem0 & 1023u) != 0;  // the swizzled tiles need the declared alignment

  if (warp == kFewMMA) tc::tmem_alloc<kFewTmem>(smem_u32(tmem_slot));
  if (tid == 0) {
    for (int st = 0; st < p.stages; ++st) {
      tc::mbar_init(bar0 + 8 * (kFullBar + st), 1);
      tc::mbar_init(bar0 + 8 * (kEmptyBar + st), 1);
    }
    tc::mbar_init(bar0 + 8 * kDoneBar, 1);
    tc::mbar_init_fence();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();

  float* part = reinterpret_cast<float*>(smem);  // [TN][128] partial results, over the ring
  if (warp == kFewCOPY) {
    if (lane == 0 && !bad) {
      int st = 0;
      uint32_t ph = 0, first = 1;
      for (int c = c0; c < c1; ++c) {
        if (!first && !wait(bar0 + 8 * (kEmptyBar + st), ph ^ 1, p.wait_ns)) {
          bad = 1;
          break;
        }
        const uint32_t base = smem0 + st * p.stage_bytes, fb = bar0 + 8 * (kFullBar + st);
        tc::mbar_expect_tx(fb, p.stage_bytes);
        if constexpr (WMN) {
          load_3d<1>(base, &w_map, n0, c * kKC, 0, fb);
          load_3d<1>(base + 8192, &w_map, n0 + 64, c * kKC, 0, fb);
        } else {
          load_3d<1>(base, &w_map, c * kKC, n0, 0, fb);
        }
        load_3d<1>(base + kABytes, &x_map, c * kKC, t00, 0, fb);
        if (++st == p.stages) {
          st = 0;
          ph ^= 1;
          first = 0;
        }
      }
      // every load issued has landed before the ring is written over
      for (int s2 = 0; s2 < (first ? st : p.stages); ++s2)
        wait(bar0 + 8 * (kFullBar + s2), s2 < st ? ph : ph ^ 1, p.wait_ns);
    }
    __syncwarp();
  } else if (warp == kFewMMA) {
    if (!bad) {
      constexpr uint32_t kHi = desc_hi(1024, kSW128), kAStep = (WMN ? 2048 : 32) >> 4;
      const uint32_t a0 = desc_lo(smem0, WMN ? 8192 : 16), b0 = desc_lo(smem0 + kABytes, 16);
      const uint32_t stage_step = p.stage_bytes >> 4, idesc = p.idesc;
      int st = 0;
      uint32_t ph = 0;
      for (int c = c0; c < c1; ++c) {
        if (!warp_wait(bar0 + 8 * (kFullBar + st), ph, p.wait_ns)) {
          bad = 1;
          break;
        }
        tc::fence_after_sync();
        const uint32_t a = a0 + st * stage_step, b = b0 + st * stage_step;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma<1>(tmem, a + kk * kAStep, kHi, b + kk * 2, kHi, idesc, c > c0 || kk > 0);
          tc::commit(bar0 + 8 * (kEmptyBar + st));
        }
        __syncwarp();
        if (++st == p.stages) {
          st = 0;
          ph ^= 1;
        }
      }
#ifdef SWIN_WATTN_FAULT_INJECTION
      if (p.fault != kFaultGemm)
#endif
        if (elect_one()) tc::commit(bar0 + 8 * kDoneBar);
      __syncwarp();
      if (!warp_wait(bar0 + 8 * kDoneBar, 0, p.wait_ns)) bad = 1;
    }
  }
  // the MMAs have read the last stages and every load has landed: the ring is free
  __syncthreads();
  if (warp < kFewEpi) {
    if (!warp_wait(bar0 + 8 * kDoneBar, 0, p.wait_ns)) bad = 1;
    if (!bad) {
      tc::fence_after_sync();
      const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      for (int t = (warp >> 2) * 16; t < p.TN; t += kFewEpi / 4 * 16) {
        uint32_t a[16];
        tc::ld16_wait(trow + t, a);
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(t + e) * kBM + (tid & (kBM - 1))] = __uint_as_float(a[e]);
      }
    }
    tc::fence_before_sync();
  }
  if (S > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // This CTA finishes the tokens rank, rank + S, ... of the tile: four warps per 32 output
  // channels in turn, kBatch tokens at a time with their loads in flight together.
  if (!bad) {
    constexpr int kBatch = 8;
    const int n = n0 + (tid & (kBM - 1));
    if (warp < kFewEpi && n < p.N) {
      const float bias = EPI == kEpiAct && p.bias != nullptr ? p.bias[n] : 0.0f;
      const uint32_t mine = smem0 + (n - n0) * 4;
      uint32_t peer[kMaxCluster];
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s) peer[s] = map_to_rank(mine, s < S ? s : 0);
      const int step = kFewEpi / 4 * S;
      for (int t0 = rank + (warp >> 2) * S; t0 < tokens; t0 += kBatch * step) {
        float aux[kBatch], acc[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int t = t0 + u * step;
          aux[u] = p.aux != nullptr && t < tokens ? bf16_value(p.aux + (int64_t)(t00 + t) * p.N + n) : 0.0f;
          acc[u] = 0.0f;
        }
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
          if (s < S) {
            float v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              v[u] = 0.0f;
              if (t0 + u * step < tokens) v[u] = load_cluster(peer[s] + (t0 + u * step) * (kBM * 4));
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) acc[u] += v[u];
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int t = t0 + u * step;
          if (t < tokens) {
            const int64_t at = (int64_t)(t00 + t) * p.N + n;
            float z = 0.0f;
            const float y = finish<EPI>(acc[u], bias, aux[u], p.act, &z);
            p.out[at] = __float2bfloat16_rn(y);
            if (EPI == kEpiAct && p.pre != nullptr) p.pre[at] = __float2bfloat16_rn(z);
          }
        }
      }
    }
  }
  if (bad && p.status != nullptr) atomicOr(p.status, 1);
  // no CTA leaves while another reads its partial results
  if (S > 1)
    cluster_sync_all();
  else
    __syncthreads();
  if (warp == kFewMMA) tc::tmem_dealloc<kFewTmem>(tmem);
}

template <bool WMN, int EPI>
cudaError_t launch_few(const FewTiling& t, const Matrix& w, const Matrix& x, FewParams p, cudaStream_t st) {
  constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr CUtensorMapL2promotion kL2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  p.TN = t.TN;
  p.n_tiles = t.n_tiles;
  p.chunks = t.chunks;
  p.cluster = t.cluster;
  CUtensorMap w_map, x_map;
  cudaError_t e = encode_3d(&w_map, w, 1, kBf16, 2, kKC, WMN ? 64 : kBM, CU_TENSOR_MAP_SWIZZLE_128B, kL2);
  if (e == cudaSuccess) e = encode_3d(&x_map, x, 1, kBf16, 2, kKC, p.TN, CU_TENSOR_MAP_SWIZZLE_128B, kL2);
  DeviceInfo di;
  if (e == cudaSuccess) e = device_info(&di);
  if (e != cudaSuccess) return e;
  p.wait_ns = wait_limit_ns();
  p.fault = fault_site();
  p.idesc = tc::idesc_bf16(kBM, p.TN, false, WMN);
  p.stage_bytes = kABytes + p.TN * 128;
  constexpr int kFixed = 8 * kFewBars + 16;
  p.stages = std::min(kMaxStages, (di.smem_max - kFixed) / p.stage_bytes);
  if (p.stages < 2) return cudaErrorInvalidConfiguration;
  p.off_bar = std::max(p.stages * p.stage_bytes, p.TN * kBM * 4);
  // more than half of an SM's shared memory: one CTA per SM, so the tensor memory is free
  const int smem = std::max(120 * 1024, p.off_bar + kFixed);
  auto kern = few_kernel<WMN, EPI>;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(reinterpret_cast<const void*>(kern), di.smem_max, di.device, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(t.n_tiles * t.t_tiles * t.cluster));
  cfg.blockDim = dim3(kFewWarps * 32);
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
  return cudaLaunchKernelEx(&cfg, kern, w_map, x_map, p);
}

}  // namespace

FewTiling few_tiling(int64_t T, int N, int64_t K) {
  FewTiling t;
  t.t_tiles = (int)((T + kMaxTN - 1) / kMaxTN);
  t.TN = (int)((T + t.t_tiles - 1) / t.t_tiles + 15) / 16 * 16;
  t.n_tiles = (N + kBM - 1) / kBM;
  t.chunks = (int)((K + kKC - 1) / kKC);
  t.cluster = 1;
  const int64_t tiles = (int64_t)t.n_tiles * t.t_tiles;
  for (int s = 2; s <= kMaxCluster; ++s)
    if (tiles <= kResidentClusters[s] && t.chunks >= 2 * s) t.cluster = s;
  const double chunks = (t.chunks + t.cluster - 1) / t.cluster;
  const double rounds = (double)((tiles + kResidentClusters[t.cluster] - 1) / kResidentClusters[t.cluster]);
  t.cost = 7000.0 + rounds * (chunks * std::max(200.0, 2.4 * (kBM + t.TN)) + 500.0 * t.cluster + 40.0 * t.TN);
  return t;
}

cudaError_t linear_few_launch(const FewTiling& t, const void* x, const void* w, const float* b, const void* residual, void* y, void* pre,
                              int T, int K, int N, int act, int* status, cudaStream_t st) {
  FewParams p{};
  p.T = T;
  p.N = N;
  p.act = act;
  p.bias = b;
  p.aux = static_cast<const __nv_bfloat16*>(residual);
  p.out = static_cast<__nv_bfloat16*>(y);
  p.pre = static_cast<__nv_bfloat16*>(pre);
  p.status = status;
  return launch_few<false, kEpiAct>(t, Matrix{w, N, K, K, 0}, Matrix{x, T, K, K, 0}, p, st);
}

cudaError_t linear_bwd_data_few_launch(const FewTiling& t, const void* dy, const void* w, const void* pre, void* dx, int T, int K, int N,
                                       int act, int* status, cudaStream_t st) {
  FewParams p{};
  p.T = T;
  p.N = K;
  p.act = act;
  p.aux = act == SWIN_WATTN_ACT_NONE ? nullptr : static_cast<const __nv_bfloat16*>(pre);
  p.out = static_cast<__nv_bfloat16*>(dx);
  p.status = status;
  return launch_few<true, kEpiSlope>(t, Matrix{w, N, K, K, 0}, Matrix{dy, T, N, N, 0}, p, st);
}

}  // namespace swin
