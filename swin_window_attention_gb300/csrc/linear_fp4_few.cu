// The 4-bit dense layer (linear_fp4.cu) for few tokens: bound by reading the weight, and by latency. As in the 16-bit
// form (linear_few.cu) the weight's rows are the MMA's 128 rows and the tokens its N, and a cluster of up to eight CTAs
// shares a tile, each over its part of K; their partial results are summed in order through distributed
// shared memory. What differs:
// * x is quantised here: the epilogue's warps, idle until then, bring each chunk of x [tokens, 256] as it lies (or its
//   codes and scales, where it is quantised already), and write codes and scales into shared memory as the tensor core
//   reads them. One launch then does what takes two, and no workspace is read back.
// * a chunk is 256 elements, its scales go through tensor memory.
#include "fp4_quantize.cuh"
#include "linear_fp4.cuh"

namespace swin {

namespace {

using namespace prod;

constexpr int kEpi = 16, kMma = kEpi, kCopy = kEpi + 1, kWarps = kEpi + 2;
constexpr int kMaxCluster4 = 8, kMaxTN4 = 128, kMaxRing = 8;
constexpr int kFullB = 0, kEmptyB = kMaxRing, kDoneB = 2 * kMaxRing, kBarsF = kDoneB + 1;
// Tensor memory: the accumulator, then two sets of scales, of the weight and of the tokens.
constexpr int kTmem = 256, kScaleCol = kMaxTN4, kSetCol = 32, kScaleOfX = 16;

struct FewFp4Params {
  int T, N, K, TN;  // tokens, result columns, tokens per tile (the MMA's N)
  int n_tiles;      // tiles along N
  int chunks, steps, k_tiles;
  int cluster;
  int stages, stage_bytes, off_x, off_sw, off_sx, off_bar;
  uint32_t idesc;
  int act;
  const void* x;  // bf16 or fp32, or codes
  const unsigned char *x_scales, *w_scales;
  const float *scale_x, *scale_w;
  const float* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  int* status;
  uint64_t wait_ns;
  int fault;
};

__device__ __forceinline__ float load_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float activate(float z, int act) {
  const float2 v = make_float2(z, 0.0f);
  switch (act) {
    case SWIN_WATTN_ACT_RELU: return act_value<SWIN_WATTN_ACT_RELU>(v).x;
    case SWIN_WATTN_ACT_GELU: return act_value<SWIN_WATTN_ACT_GELU>(v).x;
    case SWIN_WATTN_ACT_GELU_TANH: return act_value<SWIN_WATTN_ACT_GELU_TANH>(v).x;
    case SWIN_WATTN_ACT_SILU: return act_value<SWIN_WATTN_ACT_SILU>(v).x;
  }
  return z;
}

// A chunk of x in a stage: row t of the codes at 128 t, its 16-byte pieces swizzled as the copy engine would; the scale of
// row t and block j of a tile at (t % 32) * 16 + (t / 32) * 4 + j.

// Codes and scales of chunk c, by asynchronous copies: 8 pieces of 16 bytes a token, then its scale words.
template <int FORMAT>
__device__ __forceinline__ void fetch_codes(const FewFp4Params& p, uint32_t codes, uint32_t scales, int c, int t00, int tokens,
                                            int tid) {
  constexpr int kTPC = fp4::chunk_tiles(FORMAT);
  const int64_t row_bytes = p.K / 2;
  const unsigned char* from = static_cast<const unsigned char*>(p.x) + t00 * row_bytes + c * 128;
  for (int i = tid; i < tokens * 8; i += kEpi * 32) {
    const int t = i >> 3, piece = i & 7;
    // (past the end of a row: zero bytes are read, the rest of the 16 filled with zeros)
    const int valid = c * 128 + piece * 16 < row_bytes ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(codes + t * 128 + ((piece ^ (t & 7)) << 4)),
                 "l"(valid != 0 ? from + t * row_bytes + piece * 16 : from), "r"(valid)
                 : "memory");
  }
  for (int i = tid; i < tokens * kTPC; i += kEpi * 32) {
    const int t = i / kTPC, k = i % kTPC;
    if (c * kTPC + k < p.k_tiles)  // (tiles past the end have no step)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(scales + k * fp4::kTileBytes + (t & 31) * 16 + (t >> 5) * 4),
                   "l"(p.x_scales + fp4::scale_word(t00 + t, c * kTPC + k, p.k_tiles))
                   : "memory");
  }
  cp_async_commit();
}

// Unit i of chunk c, 16 elements of token i / 16, as it lies in memory (past the end of a row nothing).
template <typename T>
__device__ __forceinline__ fp4::Raw16<T> read_unit(const FewFp4Params& p, int c, int i, int t00) {
  const int t = i >> 4, k = c * 256 + (i & 15) * 16;
  fp4::Raw16<T> raw{};
  if (k < p.K) raw = fp4::load16(static_cast<const T*>(p.x) + (int64_t)(t00 + t) * p.K + k);
  return raw;
}
// The same, quantised, into a stage. A block of MXFP4 is two neighbouring threads' (K is a multiple of 32: both or neither
// past the end, where zeros give codes and a scale of zero).
template <typename T, int FORMAT>
__device__ __forceinline__ void write_unit(const fp4::Raw16<T>& raw, unsigned char* codes, unsigned char* scales, int i, float ts,
                                           float r_ts) {
  const int t = i >> 4, u = i & 15, j = FORMAT == 0 ? u : u >> 1;
  uint32_t scale;
  const uint2 q = fp4::quantize16<FORMAT>(raw, ts, r_ts, 3u << (threadIdx.x & 30), scale);
  *reinterpret_cast<uint2*>(codes + t * 128 + (((u >> 1) ^ (t & 7)) << 4) + (u & 1) * 8) = q;
  if (FORMAT == 0 || (u & 1) == 0)
    scales[(j >> 2) * fp4::kTileBytes + (t & 31) * 16 + (t >> 5) * 4 + (j & 3)] = (unsigned char)scale;
}

template <typename T, int FORMAT>
__global__ void __launch_bounds__(kWarps * 32, 1)
    few_fp4_kernel(const __grid_constant__ CUtensorMap w_map, const FewFp4Params p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  constexpr int kTPC = fp4::chunk_tiles(FORMAT);
  pdl_launch_dependents();
  const uint32_t smem0 = smem_u32(smem), bar0 = smem0 + p.off_bar;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // cluster -> 128 output channels from n0 of the TN tokens from t00
  const int S = p.cluster, rank = blockIdx.x % S, tile = blockIdx.x / S;
  const int n0 = tile % p.n_tiles * kBM, t00 = tile / p.n_tiles * p.TN, tokens = min(p.TN, p.T - t00);
  // this CTA's chunks of K
  const int c0 = (int)((int64_t)p.chunks * rank / S), c1 = (int)((int64_t)p.chunks * (rank + 1) / S);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + p.off_bar + 8 * kBarsF);
  int bad = (smem0 & 1023u) != 0;  // the swizzled tiles need the declared alignment

  if (warp == kMma) tc::tmem_alloc<kTmem>(smem_u32(tmem_slot));
  if (tid == 0) {
    for (int st = 0; st < p.stages; ++st) {
      tc::mbar_init(bar0 + 8 * (kFullB + st), 1 + kEpi);  // the copy warp and those that bring x
      tc::mbar_init(bar0 + 8 * (kEmptyB + st), 1);
    }
    tc::mbar_init(bar0 + 8 * kDoneB, 1);
    tc::mbar_init_fence();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();

  float* part = reinterpret_cast<float*>(smem);  // [TN][128] partial results, over the ring
  if (warp == kCopy) {
    if (lane == 0 && !bad) {
      int st = 0;
      uint32_t ph = 0, first = 1;
      for (int c = c0; c < c1; ++c) {
        if (!first && !wait(bar0 + 8 * (kEmptyB + st), ph ^ 1, p.wait_ns)) {
          bad = 1;
          break;
        }
        const uint32_t base = smem0 + st * p.stage_bytes, fb = bar0 + 8 * (kFullB + st);
        const int tiles = min(kTPC, p.k_tiles - c * kTPC);
        tc::mbar_expect_tx(fb, kABytes + tiles * fp4::kTileBytes);
        load_3d<1>(base, &w_map, c * 128, n0, 0, fb);
        tc::bulk_copy(base + p.off_sw, p.w_scales + ((int64_t)(n0 >> 7) * p.k_tiles + c * kTPC) * fp4::kTileBytes,
                      tiles * fp4::kTileBytes, fb);
        if (++st == p.stages) {
          st = 0;
          ph ^= 1;
          first = 0;
        }
      }
      // every load issued has landed before the ring is written over
      for (int s2 = 0; s2 < (first ? st : p.stages); ++s2)
        wait(bar0 + 8 * (kFullB + s2), s2 < st ? ph : ph ^ 1, p.wait_ns);
    }
    __syncwarp();
  } else if (warp == kMma) {
    if (!bad) {
      constexpr uint32_t kHi = desc_hi(1024, kSW128);
      const uint32_t a0 = desc_lo(smem0, 16), b0 = desc_lo(smem0 + p.off_x, 16), stage_step = p.stage_bytes >> 4;
      const uint32_t sa0 = fp4::scale_lo(smem0 + p.off_sw), sb0 = fp4::scale_lo(smem0 + p.off_sx);
      const uint32_t id0 = p.idesc, id1 = p.idesc | fp4::idesc_second_half();
      int st = 0, set = 0;
      uint32_t ph = 0;
      for (int c = c0; c < c1; ++c) {
        if (!warp_wait(bar0 + 8 * (kFullB + st), ph, p.wait_ns)) {
          bad = 1;
          break;
        }
        tc::fence_after_sync();
        const uint32_t at = st * stage_step;
        const uint32_t sa = tmem + kScaleCol + set * kSetCol, sb = sa + kScaleOfX;
        const int steps = min(4, p.steps - 4 * c);
        if (elect_one()) {
          for (int k = 0; k * (4 / kTPC) < steps; ++k) {
            fp4::copy_scales<1>(sa + 4 * k, sa0 + at + k * (fp4::kTileBytes >> 4));
            fp4::copy_scales<1>(sb + 4 * k, sb0 + at + k * (fp4::kTileBytes >> 4));
          }
          for (int kk = 0; kk < steps; ++kk) {
            const int k = kk / (4 / kTPC);
            fp4::mma<1, FORMAT>(tmem, a0 + at + kk * 2, b0 + at + kk * 2, kHi, FORMAT == 1 && (kk & 1) ? id1 : id0, sa + 4 * k,
                                sb + 4 * k, c > c0 || kk > 0);
          }
          tc::commit(bar0 + 8 * (kEmptyB + st));
        }
        __syncwarp();
        set ^= 1;
        if (++st == p.stages) {
          st = 0;
          ph ^= 1;
        }
      }
#ifdef SWIN_WATTN_FAULT_INJECTION
      if (p.fault != kFaultGemm)
#endif
        if (elect_one()) tc::commit(bar0 + 8 * kDoneB);
      __syncwarp();
      if (!warp_wait(bar0 + 8 * kDoneB, 0, p.wait_ns)) bad = 1;
    }
  } else if (!bad) {
    int st = 0;
    uint32_t ph = 0, first = 1;
    auto next_stage = [&](int& stage) {
      if (++stage == p.stages) stage = 0;
      return stage == 0;
    };
    auto hand_over = [&](int stage) {
      tc::fence_proxy_async();  // the tensor core reads what these threads wrote
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar0 + 8 * (kFullB + stage));
    };
    if constexpr (sizeof(T) == 1) {
      int done = 0, behind = 0;  // the stage to hand over next; chunks on their way
      for (int c = c0; c < c1; ++c) {
        if (!first && !warp_wait(bar0 + 8 * (kEmptyB + st), ph ^ 1, p.wait_ns)) {
          bad = 1;
          break;
        }
        const uint32_t base = smem0 + st * p.stage_bytes;
        fetch_codes<FORMAT>(p, base + p.off_x, base + p.off_sx, c, t00, tokens, tid);
        if (next_stage(st)) {
          ph ^= 1;
          first = 0;
        }
        if (++behind > 2) {  // (there are four stages at least)
          cp_async_wait<2>();
          hand_over(done);
          next_stage(done);
          --behind;
        }
      }
      cp_async_wait_all();
      for (; behind > 0; --behind) {
        hand_over(done);
        next_stage(done);
      }
    } else {
      // a thread's units of all chunks in turn, the next one on its way
      const float ts = FORMAT == 0 ? *p.scale_x : 1.0f, r_ts = fp4::reciprocal(ts);
      const int units = tokens * 16;
      auto next_unit = [&](int& c, int& i) {
        i += kEpi * 32;
        if (i >= units) {
          i = tid;
          ++c;
        }
      };
      int ca = c0, ia = tid;  // the unit ahead
      fp4::Raw16<T> ahead{};
      if (tid < units) {
        ahead = read_unit<T>(p, ca, ia, t00);
        next_unit(ca, ia);
      }
      for (int c = c0; c < c1; ++c) {
        if (!first && !warp_wait(bar0 + 8 * (kEmptyB + st), ph ^ 1, p.wait_ns)) {
          bad = 1;
          break;
        }
        unsigned char* base = smem + st * p.stage_bytes;
        for (int i = tid; i < units; i += kEpi * 32) {
          const fp4::Raw16<T> raw = ahead;
          if (ca < c1) {
            ahead = read_unit<T>(p, ca, ia, t00);
            next_unit(ca, ia);
          }
          write_unit<T, FORMAT>(raw, base + p.off_x, base + p.off_sx, i, ts, r_ts);
        }
        hand_over(st);
        if (next_stage(st)) {
          ph ^= 1;
          first = 0;
        }
      }
    }
  }
  // the MMAs have read the last stages and every load has landed: the ring is free
  __syncthreads();
  // (the tensors' scales are used up here as far as fp32 does not hold their product: a branch in the batches below cost 49
  // tokens half a microsecond)
  float2 scales = make_float2(1.0f, 1.0f);
  if (warp < kEpi) {
    if constexpr (FORMAT == 0) scales = fp4::tensor_scales(*p.scale_x, *p.scale_w);
    if (!warp_wait(bar0 + 8 * kDoneB, 0, p.wait_ns)) bad = 1;
    if (!bad) {
      tc::fence_after_sync();
      const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      for (int t = (warp >> 2) * 16; t < p.TN; t += kEpi / 4 * 16) {
        uint32_t a[16];
        tc::ld16_wait(trow + t, a);
        if (scales.x != 1.0f) {
#pragma unroll
          for (int e = 0; e < 16; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * scales.x);
        }
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
  // This CTA finishes the tokens rank, rank + S, ... of the tile: four warps per 32 output channels in turn, kBatch
  // tokens at a time with their loads in flight together.
  if (!bad) {
    constexpr int kBatch = 8;
    const int n = n0 + (tid & (kBM - 1));
    if (warp < kEpi && n < p.N) {
      const float bias = p.bias != nullptr ? p.bias[n] : 0.0f;
      const float scale = scales.y;
      const uint32_t mine = smem0 + (n - n0) * 4;
      uint32_t peer[kMaxCluster4];
#pragma unroll
      for (int s = 0; s < kMaxCluster4; ++s) peer[s] = map_to_rank(mine, s < S ? s : 0);
      const int step = kEpi / 4 * S;
      for (int t0 = rank + (warp >> 2) * S; t0 < tokens; t0 += kBatch * step) {
        float more[kBatch], acc[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int t = t0 + u * step;
          more[u] = p.residual != nullptr && t < tokens ? __bfloat162float(p.residual[(int64_t)(t00 + t) * p.N + n]) : 0.0f;
          acc[u] = 0.0f;
        }
#pragma unroll
        for (int s = 0; s < kMaxCluster4; ++s) {
          if (s < S) {
            float v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              v[u] = 0.0f;
              if (t0 + u * step < tokens) v[u] = load_peer(peer[s] + (t0 + u * step) * (kBM * 4));
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) acc[u] += v[u];
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int t = t0 + u * step;
          if (t < tokens)
            p.out[(int64_t)(t00 + t) * p.N + n] = __float2bfloat16_rn(activate(fmaf(acc[u], scale, bias), p.act) + more[u]);
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
  if (warp == kMma) tc::tmem_dealloc<kTmem>(tmem);
}

template <typename T, int FORMAT>
cudaError_t launch_few4(const FewFp4Tiling& t, const Fp4Operand& w, FewFp4Params p, cudaStream_t st) {
  CUtensorMap w_map;
  cudaError_t e = fp4::encode_codes(&w_map, w, p.N, p.K, kBM);
  DeviceInfo di;
  if (e == cudaSuccess) e = device_info(&di);
  if (e != cudaSuccess) return e;
  constexpr int kSetBytes = fp4::chunk_tiles(FORMAT) * fp4::kTileBytes;
  p.TN = t.TN;
  p.n_tiles = t.n_tiles;
  p.chunks = t.chunks;
  p.cluster = t.cluster;
  p.steps = (p.K + fp4::kStep - 1) / fp4::kStep;
  p.k_tiles = fp4::k_tiles(p.K, FORMAT);
  p.w_scales = static_cast<const unsigned char*>(w.scales);
  p.scale_w = w.tensor_scale;
  p.wait_ns = wait_limit_ns();
  p.fault = fault_site();
  p.idesc = fp4::idesc(kBM, p.TN, FORMAT);
  p.off_x = kABytes;
  p.off_sw = p.off_x + p.TN * 128;
  p.off_sx = p.off_sw + kSetBytes;
  p.stage_bytes = (p.off_sx + kSetBytes + 1023) / 1024 * 1024;
  constexpr int kFixed = 8 * kBarsF + 16;
  p.stages = std::min(kMaxRing, (di.smem_max - kFixed) / p.stage_bytes);
  if (p.stages < 2) return cudaErrorInvalidConfiguration;
  p.off_bar = std::max(p.stages * p.stage_bytes, p.TN * kBM * 4);
  // more than half of an SM's shared memory: one CTA per SM, so the tensor memory is free
  const int smem = std::max(120 * 1024, p.off_bar + kFixed);
  auto kern = few_fp4_kernel<T, FORMAT>;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(reinterpret_cast<const void*>(kern), di.smem_max, di.device, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(t.n_tiles * t.t_tiles * t.cluster));
  cfg.blockDim = dim3(kWarps * 32);
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
  return cudaLaunchKernelEx(&cfg, kern, w_map, p);
}

}  // namespace

FewFp4Tiling few_fp4_tiling(int64_t T, int N, int K) {
  FewFp4Tiling t;
  t.t_tiles = (int)((T + kMaxTN4 - 1) / kMaxTN4);
  t.TN = (int)((T + t.t_tiles - 1) / t.t_tiles + 15) / 16 * 16;
  t.n_tiles = (N + kBM - 1) / kBM;
  t.chunks = (K + fp4::kChunk - 1) / fp4::kChunk;
  t.cluster = 1;
  const int64_t tiles = (int64_t)t.n_tiles * t.t_tiles;
  for (int s = 2; s <= kMaxCluster4; ++s)
    if (tiles <= kResidentClusters[s] && t.chunks >= s) t.cluster = s;
  const double rounds = (double)((tiles + kResidentClusters[t.cluster] - 1) / kResidentClusters[t.cluster]);
  t.chunk_rounds = rounds * ((t.chunks + t.cluster - 1) / t.cluster);
  t.cost = 6300.0 + 800.0 * t.chunk_rounds +
           rounds * ((t.cluster > 1 ? 1000.0 + 200.0 * t.cluster : 0.0) + 40.0 * t.TN / t.cluster);
  return t;
}

cudaError_t linear_fp4_few_launch(const FewFp4Tiling& t, const void* x, const void* x_scales, int x_bytes, const float* x_scale,
                                  const Fp4Operand& w, const float* b, const void* residual, void* y, int T, int K, int N,
                                  int format, int act, int* status, cudaStream_t st) {
  FewFp4Params p{};
  p.T = T;
  p.N = N;
  p.K = K;
  p.act = act;
  p.x = x;
  p.x_scales = static_cast<const unsigned char*>(x_scales);
  p.scale_x = x_scale;
  p.bias = b;
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.out = static_cast<__nv_bfloat16*>(y);
  p.status = status;
  switch (x_bytes * 2 + format) {
    case 1 * 2 + 0: return launch_few4<uint8_t, 0>(t, w, p, st);
    case 1 * 2 + 1: return launch_few4<uint8_t, 1>(t, w, p, st);
    case 2 * 2 + 0: return launch_few4<__nv_bfloat16, 0>(t, w, p, st);
    case 2 * 2 + 1: return launch_few4<__nv_bfloat16, 1>(t, w, p, st);
    case 4 * 2 + 0: return launch_few4<float, 0>(t, w, p, st);
    default: return launch_few4<float, 1>(t, w, p, st);
  }
}

}  // namespace swin
