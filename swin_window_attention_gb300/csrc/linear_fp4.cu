// A dense layer on microscaled 4-bit operands (fp4.cuh):
//   y = residual + act(ts_x ts_w sum_k (q_x s_x)(q_w s_w) + b)
// The block-scaled MMAs multiply 4-bit elements and apply both operands' block scales in the tensor core,
// accumulating in fp32; the scales of the tensors multiply the sum once, in the epilogue.
//
// One persistent CTA per SM (CG = 1) or pair of CTAs on two SMs (CG = 2) walks output tiles of CG * 128 tokens by
// NT <= 192 channels, as the 16-bit products do (product.cuh):
// * copy warp: per chunk of 256 along K, 128 rows of x and NT / CG of w (128 bytes each) into a ring of stages;
// * scale warp: their scale tiles into the same stages;
// * MMA warp: the chunk's scales from shared to tensor memory (two sets of columns in turn), and four MMAs
//   of K = 64 into one of two accumulators;
// * sixteen epilogue warps: 32-column slices, arithmetic in fp32, one rounding, TMA stores; a residual arrives by
//   TMA in the staging tile that its result is written over.
// Every wait is bounded (1 s); a wait that runs out sets the caller's status word and the CTA leaves after its
// copies have landed and its tensor memory is freed.
#include "linear_fp4.cuh"

namespace swin {

namespace {

using namespace prod;

constexpr int kEpiWarps = 16, kMMA = kEpiWarps, kCOPY = kEpiWarps + 1, kSCALES = kEpiWarps + 2, kNThreads = (kEpiWarps + 3) * 32;
constexpr int kMaxNT4 = 192, kSlices4 = 3;  // slices of a warp: six of a tile between at least two warps
// Tensor memory: two accumulators, then two sets of scales: A's four tiles, B's four times two.
constexpr int kScaleCols = 2 * kMaxNT4, kSetCols = 48, kScaleB = 16;
constexpr int kMaxTiles = 4;  // staging tiles of an epilogue warp
constexpr int kTile = 2048;   // 32 rows x 32 columns of bf16
constexpr int kFull = 0, kEmpty = kMaxStages, kDFull4 = 2 * kMaxStages, kDFree4 = kDFull4 + 2, kDrain4 = kDFree4 + 2,
              kAux4 = kDrain4 + 1, kBars = kAux4 + kMaxTiles * kEpiWarps;

struct Fp4Params {
  int M, N, NT;
  FastDiv n_nt;
  int n_items;  // tiles, along N fastest
  int chunks, steps;  // of K, in 256 and in 64
  const unsigned char *scales_a, *scales_b;
  int k_tiles;  // scale tiles along K
  int stages, stage_bytes, off_sa, off_sb, b_tiles;  // b_tiles: scale row tiles of B a stage holds
  int off_out, warp_bytes, tiles, off_bias, off_bar;
  int per_quad;  // epilogue warps of a quadrant of lanes that have slices
  uint32_t idesc;
  int act;
  bool has_aux;
  const float* bias;
  const float *scale_x, *scale_w;  // of the tensors, or null
  int* status;
  uint64_t wait_ns;
  int fault;
};

template <int CG, int FORMAT>
__global__ void __launch_bounds__(kNThreads, 1)
    linear_fp4_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                      const __grid_constant__ CUtensorMap out_map, const __grid_constant__ CUtensorMap aux_map,
                      const Fp4Params p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  constexpr int kTPC = fp4::chunk_tiles(FORMAT), kSetBytes = kTPC * fp4::kTileBytes;
  pdl_launch_dependents();
  const uint32_t smem0 = smem_u32(smem);
  if ((smem0 & 1023u) != 0) {  // the swizzled tiles need the declared alignment
    if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, 1);
    return;
  }
  const uint32_t bar0 = smem0 + p.off_bar;
  auto full_bar = [&](int st) { return bar0 + 8 * (kFull + st); };
  auto empty_bar = [&](int st) { return bar0 + 8 * (kEmpty + st); };
  auto dfull_bar = [&](int b) { return bar0 + 8 * (kDFull4 + b); };
  auto dfree_bar = [&](int b) { return bar0 + 8 * (kDFree4 + b); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + p.off_bar + 8 * kBars);
  const int stages = p.stages;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = CG == 2 ? (int)cluster_rank() : 0;
  const int group = blockIdx.x / CG, n_groups = gridDim.x / CG;
  auto rows_of_item = [&](int it, int& m0, int& n0) {
    const uint32_t mt = p.n_nt.quotient(it);
    m0 = ((int)mt * CG + rank) * kBM;
    n0 = (it - (int)mt * (int)p.n_nt.d) * p.NT;
  };

  if (warp == kMMA) tmem_alloc<CG>(smem_u32(tmem_slot));
  if (tid == 0) {
    for (int st = 0; st < stages; ++st) {
      tc::mbar_init(full_bar(st), 1 + CG);  // the codes of both CTAs and the scales of each
      tc::mbar_init(empty_bar(st), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(dfull_bar(b), 1);
      tc::mbar_init(dfree_bar(b), kEpiWarps * CG);
    }
    tc::mbar_init(bar0 + 8 * kDrain4, 1);
    for (int b = 0; b < kMaxTiles * kEpiWarps; ++b) tc::mbar_init(bar0 + 8 * (kAux4 + b), 1);
    tc::mbar_init_fence();
  }
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // The prologue above touches only this CTA's shared and tensor memory, so it may overlap
  // the previous kernel on the stream; every global access comes after this wait.
  pdl_wait();
  int bad = 0;
  if (warp == kCOPY) {
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0, first = 1;
      // a pair's loads all complete on the first CTA's barriers
      const uint32_t full0 = CG == 2 ? map_to_rank(full_bar(0), 0) : full_bar(0);
      for (int it = group; it < p.n_items && !bad; it += n_groups) {
        int m0, n0;
        rows_of_item(it, m0, n0);
        for (int c = 0; c < p.chunks; ++c) {
          if (!first && !wait(empty_bar(st), ph ^ 1, p.wait_ns)) {
            bad = 1;
            break;
          }
          const uint32_t base = smem0 + st * p.stage_bytes, fb = full0 + 8 * st;
          if (rank == 0) tc::mbar_expect_tx(full_bar(st), CG * (kABytes + (p.NT / CG) * 128));
          load_3d<CG>(base, &a_map, c * 128, m0, 0, fb);
          load_3d<CG>(base + kABytes, &b_map, c * 128, n0 + rank * (p.NT / CG), 0, fb);
          if (++st == stages) {
            st = 0;
            ph ^= 1;
            first = 0;
          }
        }
      }
      // every load issued has landed before the CTA leaves (the second CTA of a pair is held
      // by the cluster barrier below until the first has seen its bytes too)
      if (rank == 0)
        for (int s2 = 0; s2 < (first ? st : stages); ++s2)
          tc::mbar_wait(full_bar(s2), s2 < st ? ph : ph ^ 1, p.wait_ns);
    }
    __syncwarp();
  } else if (warp == kSCALES) {
    // The chunk's scale tiles, 16 bytes a lane: an own path beside the copy engine, whose copies cost some 100 clocks
    // each whatever their size. Chunk c is handed over once it has landed, while the next ones are on their way.
    int st = 0, done_st = 0, behind = 0;  // stages of the next chunk and of the next to hand over; chunks between them
    uint32_t ph = 0, first = 1;
    const uint32_t full0 = CG == 2 ? map_to_rank(full_bar(0), 0) : full_bar(0);
    auto hand_over = [&]() {
      tc::fence_proxy_async();  // these copies are the tensor core's to read
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          arrive_cluster(full0 + 8 * done_st);
        else
          tc::mbar_arrive(full0 + 8 * done_st);
      }
      if (++done_st == stages) done_st = 0;
      --behind;
    };
    const int row_tiles_b = (p.N + 127) >> 7, row_tiles_a = (int)(((int64_t)p.M + 127) >> 7);
    const int64_t row_bytes = (int64_t)p.k_tiles * fp4::kTileBytes;
    for (int it = group; it < p.n_items && !bad; it += n_groups) {
      int m0, n0;
      rows_of_item(it, m0, n0);
      // row tiles past the end are left as they are: their rows and columns are not stored
      const bool has_a = (m0 >> 7) < row_tiles_a, has_b1 = p.b_tiles == 2 && (n0 >> 7) + 1 < row_tiles_b;
      const unsigned char* from_a = p.scales_a + (m0 >> 7) * row_bytes + lane * 16;
      const unsigned char* from_b = p.scales_b + (n0 >> 7) * row_bytes + lane * 16;
      for (int c = 0; c < p.chunks; ++c) {
        if (!first && !warp_wait(empty_bar(st), ph ^ 1, p.wait_ns)) {
          bad = 1;
          break;
        }
        const uint32_t to = smem0 + st * p.stage_bytes + lane * 16;
#pragma unroll
        for (int k = 0; k < kTPC; ++k) {
          if (c * kTPC + k < p.k_tiles) {  // (tiles past the end have no step)
            if (has_a) cp_async_16(to + p.off_sa + k * fp4::kTileBytes, from_a + k * fp4::kTileBytes);
            cp_async_16(to + p.off_sb + k * fp4::kTileBytes, from_b + k * fp4::kTileBytes);
            if (has_b1) cp_async_16(to + p.off_sb + kSetBytes + k * fp4::kTileBytes, from_b + row_bytes + k * fp4::kTileBytes);
          }
        }
        cp_async_commit();
        from_a += kSetBytes;
        from_b += kSetBytes;
        if (++st == stages) {
          st = 0;
          ph ^= 1;
          first = 0;
        }
        // chunks on their way behind the newest: fewer than there are stages
        if (stages >= 4) {
          if (++behind > 2) {
            cp_async_wait<2>();
            hand_over();
          }
        } else if (++behind > 1) {
          cp_async_wait<1>();
          hand_over();
        }
      }
    }
    cp_async_wait_all();
    while (behind > 0) hand_over();
  } else if (warp == kMMA) {
    if (rank == 0) {
      constexpr uint32_t kHi = desc_hi(1024, kSW128);
      const uint32_t a0 = desc_lo(smem0, 16), b0 = desc_lo(smem0 + kABytes, 16), stage_step = p.stage_bytes >> 4;
      const uint32_t sa0 = fp4::scale_lo(smem0 + p.off_sa), sb0 = fp4::scale_lo(smem0 + p.off_sb);
      const uint32_t id0 = p.idesc, id1 = p.idesc | fp4::idesc_second_half();
      const int b_tiles = p.b_tiles;
      int st = 0, g = 0, set = 0;  // ring stage; accumulations begun; set of scales
      uint32_t ph = 0;
      for (int it = group; it < p.n_items && !bad; it += n_groups, ++g) {
        int m0, n0;
        rows_of_item(it, m0, n0);
        const int buf = g & 1;
        const uint32_t acc = tmem + buf * kMaxNT4;
        if (g >= 2 && !warp_wait(dfree_bar(buf), ((g >> 1) - 1) & 1, p.wait_ns)) {
          bad = 1;
          break;
        }
        for (int c = 0; c < p.chunks; ++c) {
          if (!warp_wait(full_bar(st), ph, p.wait_ns)) {
            bad = 1;
            break;
          }
          tc::fence_after_sync();
          const uint32_t at = st * stage_step, a = a0 + at, b = b0 + at, la = sa0 + at, lb = sb0 + at;
          const uint32_t sa = tmem + kScaleCols + set * kSetCols, sb = sa + kScaleB;
          const uint32_t sb_n = sb + ((n0 & 127) >> 5);  // the tile's first column may lie inside a scale tile
          const int steps = min(4, p.steps - 4 * c);
          if (elect_one()) {
            constexpr uint32_t kTileStep = fp4::kTileBytes >> 4;
            // B's tiles of one step lie side by side, four columns for 128 rows
            auto copy = [&](int k) {
              fp4::copy_scales<CG>(sa + 4 * k, la + k * kTileStep);
              fp4::copy_scales<CG>(sb + 8 * k, lb + k * kTileStep);
              if (b_tiles == 2) fp4::copy_scales<CG>(sb + 8 * k + 4, lb + (kTPC + k) * kTileStep);
            };
            auto step = [&](int kk) {
              const int k = kk / (4 / kTPC);
              fp4::mma<CG, FORMAT>(acc, a + kk * 2, b + kk * 2, kHi, FORMAT == 1 && (kk & 1) ? id1 : id0, sa + 4 * k, sb_n + 8 * k,
                                   c > 0 || kk > 0);
            };
            if (steps == 4) {
#pragma unroll
              for (int k = 0; k < kTPC; ++k) copy(k);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) step(kk);
            } else {
              for (int k = 0; k * (4 / kTPC) < steps; ++k) copy(k);
              for (int kk = 0; kk < steps; ++kk) step(kk);
            }
            commit<CG>(empty_bar(st));
#ifdef SWIN_WATTN_FAULT_INJECTION
            if (!(p.fault == kFaultGemm && g == 0))
#endif
              if (c == p.chunks - 1) commit<CG>(dfull_bar(buf));
          }
          __syncwarp();
          set ^= 1;
          if (++st == stages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      // every MMA issued has completed before the tensor memory is released
      if (elect_one()) commit_here<CG>(bar0 + 8 * kDrain4);
      __syncwarp();
      if (!warp_wait(bar0 + 8 * kDrain4, 0, p.wait_ns)) bad = 1;
    }
    __syncwarp();
  } else {
    // ==== epilogue warps ================================================================
    const int quad = warp & 3, part = warp >> 2, per_quad = p.per_quad;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
    unsigned char* wstage = smem + p.off_out + warp * p.warp_bytes;
    const bool aux = p.has_aux;
    const int NB = p.tiles;
    const uint32_t aux0 = bar0 + 8 * (kAux4 + kMaxTiles * warp);
    const float2 scales = FORMAT == 0 ? fp4::tensor_scales(*p.scale_x, *p.scale_w) : make_float2(1.0f, 1.0f);
    const float scale = scales.y;
    // the next slice whose residual is to be requested: its item and columns, and its staging tile
    int nx_it = group, nx_c0 = part * kSC, nx_end = 0, nx_row = 0, nx_n0 = 0, nx_tile = 0, issued = 0;
    auto next_item = [&]() {
      nx_end = 0;
      if (nx_it < p.n_items) {
        int m0;
        rows_of_item(nx_it, m0, nx_n0);
        nx_row = m0 + quad * 32;
        nx_end = part < per_quad && nx_row < p.M ? min(p.NT, p.N - nx_n0) : 0;
      }
    };
    auto request_next = [&]() {
      while (nx_it < p.n_items) {
        if (nx_c0 < nx_end) {
          if (lane == 0) {
            const uint32_t rb = aux0 + 8 * nx_tile;
            tc::mbar_expect_tx(rb, kTile);
            load_3d<1>(smem_u32(wstage + nx_tile * kTile), &aux_map, nx_n0 + nx_c0, nx_row, 0, rb);
          }
          ++issued;
          if (++nx_tile == NB) nx_tile = 0;
          nx_c0 += per_quad * kSC;
          return;
        }
        nx_it += n_groups;
        nx_c0 = part * kSC;
        next_item();
      }
    };
    if (aux) {
      next_item();
      for (int i = 0; i < max(NB - 2, 1); ++i) request_next();
    }
    int g = 0, m = 0, tile = 0;  // accumulations, slices of this warp, the slice's staging tile
    uint32_t aux_phase = 0;      // of that tile's barrier
    for (int it = group; it < p.n_items && !bad; it += n_groups, ++g) {
      int m0, n0;
      rows_of_item(it, m0, n0);
      const int row0 = m0 + quad * 32, buf = g & 1;
      // the bias of the tile's columns in shared memory, for broadcast reads. Every warp of a part
      // writes the same values; two buffers, and the write waits for this tile's accumulator, which is
      // given out when every warp has left the tile before last.
      float* sbias = reinterpret_cast<float*>(smem + p.off_bias) + buf * kMaxNT4 + lane;
      float bt[kSlices4];
#pragma unroll
      for (int i = 0; i < kSlices4; ++i) {
        const int c0 = (part + per_quad * i) * kSC, c = n0 + c0 + lane;
        bt[i] = p.bias != nullptr && part < per_quad && c0 < p.NT && c < p.N ? p.bias[c] : 0.0f;
      }
      if (!warp_wait(dfull_bar(buf), (g >> 1) & 1, p.wait_ns)) {
        bad = 1;
        break;
      }
      tc::fence_after_sync();
#pragma unroll
      for (int i = 0; i < kSlices4; ++i)
        if (part < per_quad && (part + per_quad * i) * kSC < p.NT) sbias[(part + per_quad * i) * kSC] = bt[i];
      __syncwarp();
#pragma unroll 1
      for (int si = 0; si < kSlices4; ++si) {
        const int c0 = (part + per_quad * si) * kSC;
        if (!(part < per_quad && row0 < p.M && c0 < p.NT && n0 + c0 < p.N)) continue;
        unsigned char* so = wstage + tile * kTile;
        if (aux) {
          // all stores but the last slice's (of two tiles, all) have read their tiles: load
          // ahead into the oldest
          if (lane == 0) {
            if (NB == 2)
              tc::bulk_wait_read<0>();
            else
              tc::bulk_wait_read<1>();
          }
          __syncwarp();
          request_next();
        }
        uint32_t a[32];
        tc::ld32_wait(trow + buf * kMaxNT4 + c0, a);
        if (scales.x != 1.0f) {
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * scales.x);
        }
        if (aux && !warp_wait(aux0 + 8 * tile, aux_phase, p.wait_ns)) {
          bad = 1;
          break;
        }
        unsigned char* sr = so + lane * 64;
        const int sw = (lane >> 1) & 3;
        auto at = [&](int c) { return reinterpret_cast<uint4*>(sr + ((c ^ sw) << 4)); };
        uint32_t o[16];  // the result, packed
        auto activate = [&](auto act) {
          constexpr int ACT = decltype(act)::value;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 r = make_uint4(0, 0, 0, 0);
            if (aux) r = *at(c);
            const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
            const float4 b0 = reinterpret_cast<const float4*>(sbias - lane + c0)[2 * c];
            const float4 b1 = reinterpret_cast<const float4*>(sbias - lane + c0)[2 * c + 1];
            const float2 bb[4] = {make_float2(b0.x, b0.y), make_float2(b0.z, b0.w), make_float2(b1.x, b1.y),
                                  make_float2(b1.z, b1.w)};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int e = 8 * c + 2 * q;
              float2 y = act_value<ACT>(__ffma2_rn(make_float2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])), splat(scale), bb[q]));
              if (aux) y = __fadd2_rn(y, unpack_bf16(rr[q]));
              o[4 * c + q] = pack_bf16(y.x, y.y);
            }
          }
        };
        switch (p.act) {
          case SWIN_WATTN_ACT_RELU: activate(std::integral_constant<int, SWIN_WATTN_ACT_RELU>()); break;
          case SWIN_WATTN_ACT_GELU: activate(std::integral_constant<int, SWIN_WATTN_ACT_GELU>()); break;
          case SWIN_WATTN_ACT_GELU_TANH: activate(std::integral_constant<int, SWIN_WATTN_ACT_GELU_TANH>()); break;
          case SWIN_WATTN_ACT_SILU: activate(std::integral_constant<int, SWIN_WATTN_ACT_SILU>()); break;
          default: activate(std::integral_constant<int, SWIN_WATTN_ACT_NONE>()); break;
        }
        if (!aux) {  // the store that held the tile has read it
          if (lane == 0) {
            if (NB == 1)
              tc::bulk_wait_read<0>();
            else
              tc::bulk_wait_read<1>();
          }
          __syncwarp();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) *at(c) = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        tc::fence_proxy_async();  // the staging tile to the copy engine
        __syncwarp();
        if (lane == 0) {
          store_3d(&out_map, n0 + c0, row0, 0, smem_u32(so));
          tc::bulk_commit();
        }
        ++m;
        if (++tile == NB) {
          tile = 0;
          aux_phase ^= 1;
        }
      }
      if (bad) break;
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          arrive_cluster(map_to_rank(dfree_bar(buf), 0));
        else
          tc::mbar_arrive(dfree_bar(buf));
      }
    }
    // after a timeout: the loads still in flight land before the CTA leaves
    for (; m < issued; ++m) {
      warp_wait(aux0 + 8 * tile, aux_phase, p.wait_ns);
      if (++tile == NB) {
        tile = 0;
        aux_phase ^= 1;
      }
    }
    if constexpr (CG == 2) cluster_arrive();  // while the last stores are written
    if (lane == 0) tc::bulk_wait_all();
  }
  if constexpr (CG == 2)
    if (warp >= kEpiWarps) cluster_arrive();
  if (bad && p.status != nullptr) atomicOr(p.status, 1);
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_wait();
  if (warp == kMMA) tmem_dealloc<CG>(tmem);
}

// ---- host side ------------------------------------------------------------------------

struct Fp4Tiling {
  int cg, NT;
  double cost;
};

// The cheapest tile by estimated clocks: rounds of tiles, each the longer of its chunks and its epilogue, plus
// one epilogue that nothing overlaps. A chunk takes 100 and a clock for each 88 of its bytes (8192^3, clocks a chunk of
// NVFP4: pairs with 192 columns 510, 128 columns 461; single SMs 609, 503); of fewer than 32 tokens, whose missing rows
// the copy engine fills in, 500 more (one token of 8192 x 8192: 18.9 us, 32 tokens: 10.4).
Fp4Tiling choose(int64_t T, int64_t N, int K, int format) {
  Fp4Tiling best{1, 64, -1.0};
  const int chunks = (K + fp4::kChunk - 1) / fp4::kChunk;
  for (int cg = 1; cg <= 2; ++cg)
    for (int nt = 64; nt <= kMaxNT4; nt += 64) {
      const int64_t items = (T + cg * kBM - 1) / (cg * kBM) * ((N + nt - 1) / nt), groups = kSms / cg;
      const double rounds = (double)((items + groups - 1) / groups);
      const int sets = fp4::chunk_tiles(format) * fp4::kTileBytes * (1 + (128 % nt != 0 ? 2 : 1));
      const double chunk = 100.0 + ((kBM + nt / cg) * 128 + sets) / 88.0 + (T < 32 ? 500.0 : 0.0), epi = 500.0 + 14.0 * nt;
      const double cost = 4000.0 + rounds * std::max(chunks * chunk, epi) + epi + (cg - 1) * 500.0;
      if (best.cost < 0.0 || cost < best.cost) best = {cg, nt, cost};
    }
  return best;
}

template <int CG, int FORMAT>
cudaError_t launch_tiles4(int NT, const Fp4Operand& x, const Fp4Operand& w, const void* residual, void* y, Fp4Params p, int K,
                          cudaStream_t st) {
  constexpr int kTPC = fp4::chunk_tiles(FORMAT), kSetBytes = kTPC * fp4::kTileBytes;
  constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap a_map, b_map, out_map, aux_map;
  cudaError_t e = fp4::encode_codes(&a_map, x, p.M, K, kBM);
  if (e == cudaSuccess) e = fp4::encode_codes(&b_map, w, p.N, K, NT / CG);
  const Matrix out{y, p.M, p.N, p.N, 0};
  if (e == cudaSuccess)
    e = encode_3d(&out_map, out, 1, kBf16, 2, kSC, 32, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
  aux_map = a_map;
  p.has_aux = residual != nullptr;
  if (e == cudaSuccess && p.has_aux)
    e = encode_3d(&aux_map, Matrix{residual, p.M, p.N, p.N, 0}, 1, kBf16, 2, kSC, 32, CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  DeviceInfo di;
  if (e == cudaSuccess) e = device_info(&di);
  if (e != cudaSuccess) return e;
  const int64_t items = ((int64_t)p.M + CG * kBM - 1) / (CG * kBM) * ((p.N + NT - 1) / NT);
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  p.NT = NT;
  p.n_nt = FastDiv((p.N + NT - 1) / NT);
  p.n_items = (int)items;
  p.steps = (K + fp4::kStep - 1) / fp4::kStep;
  p.scales_a = static_cast<const unsigned char*>(x.scales);
  p.scales_b = static_cast<const unsigned char*>(w.scales);
  p.k_tiles = fp4::k_tiles(K, FORMAT);
  p.chunks = (K + fp4::kChunk - 1) / fp4::kChunk;
  p.idesc = fp4::idesc(CG * kBM, NT, FORMAT);
  p.wait_ns = wait_limit_ns();
  p.fault = fault_site();
  // a tile that begins inside a scale tile, or is wider than one, needs two
  p.b_tiles = NT > 128 || 128 % NT != 0 ? 2 : 1;
  p.off_sa = kABytes + NT / CG * 128;
  p.off_sb = p.off_sa + kSetBytes;
  p.stage_bytes = (p.off_sb + p.b_tiles * kSetBytes + 1023) / 1024 * 1024;
  constexpr int kBiasBytes = 2 * kMaxNT4 * 4;
  // Where K is long, a tile's product takes longer than its epilogue, and shared memory is worth more in the ring: a
  // staging tile a warp, or two of half the warps where a residual comes through them. (8192^3 at five stages instead of
  // four: 192 -> 163 us NVFP4, 168 -> 158 us MXFP4; half the warps with a residual, 12561 x 6144 x 1536 54 -> 47 us, but
  // 12544 x 1536 x 6144 64 -> 70 us.)
  const bool long_k = p.chunks >= 6, longer_k = p.chunks >= 10;
  p.per_quad = p.has_aux && longer_k ? 2 : 4;
  p.tiles = p.has_aux ? (long_k ? 2 : kMaxTiles) : (long_k ? 1 : 2);
  int fixed = 0;
  for (;; --p.tiles) {  // fewer staging tiles where the ring would not have three stages
    p.warp_bytes = p.tiles * kTile;
    fixed = 4 * p.per_quad * p.warp_bytes + kBiasBytes + 8 * kBars + 16;
    p.stages = std::min(kMaxStages, (di.smem_max - fixed) / p.stage_bytes);
    if (p.stages >= 3 || p.tiles <= (p.has_aux ? 2 : 1)) break;
  }
  if (p.stages < 2) return cudaErrorInvalidConfiguration;
  p.off_out = p.stages * p.stage_bytes;
  p.off_bias = p.off_out + 4 * p.per_quad * p.warp_bytes;
  p.off_bar = p.off_bias + kBiasBytes;
  // more than half of an SM's shared memory: one CTA per SM, so the tensor memory is free
  const int smem = std::max(120 * 1024, p.off_out + fixed);
  auto kern = linear_fp4_kernel<CG, FORMAT>;
  static std::atomic<uint64_t> allowed{0};  // devices whose limit has been raised
  e = allow_smem(reinterpret_cast<const void*>(kern), di.smem_max, di.device, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(CG * std::min<int64_t>(items, di.sms / CG)));
  cfg.blockDim = dim3(kNThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a_map, b_map, out_map, aux_map, p);
}

// Above these, clusters never came out shorter.
constexpr int kFewTokens4 = 128, kFewQuantized = 64;

}  // namespace

// Whether the product itself quantises an x that is not: few tokens, of which every CTA quantises its part of K, some 400
// clocks for each 32 tokens of a chunk, against a launch of its own, some 4000 of the GPU and, where calls follow one another,
// twice as many of the host, with its workspace; counted as 6000. (In a graph, one launch and two, NVFP4 and MXFP4: one token
// 1536 -> 6144 5.1, 7.2 and 5.0, 6.6 us, 32 tokens 6.1, 7.0 and 6.4, 6.2, 49 tokens 7.3, 7.2 and 7.8, 6.5, 64 tokens 7.8, 6.9
// and 8.2, 6.2; 6144 -> 1536 one token 6.2, 7.8 and 6.0, 7.3, 64 tokens 9.2, 9.7 and 9.4, 9.0. Called from Python 49 tokens
// of MXFP4 take 19 us and 24.)
bool linear_fp4_quantizes(int T, int K, int N, int format) {
  if (T > kFewQuantized) return false;
  const FewFp4Tiling few = few_fp4_tiling(T, N, K);
  return few.cost + few.chunk_rounds * ((T + 31) / 32) * 400.0 < choose(T, N, K, format).cost + 6000.0;
}

cudaError_t linear_fp4_of_few(const void* x, int dtype, const float* x_scale, const Fp4Operand& w, const float* b,
                              const void* residual, void* y, int T, int K, int N, int format, int act, int* status,
                              cudaStream_t st) {
  return linear_fp4_few_launch(few_fp4_tiling(T, N, K), x, nullptr, dtype == SWIN_WATTN_FP32 ? 4 : 2, x_scale, w, b, residual, y,
                               T, K, N, format, act, status, st);
}

cudaError_t linear_fp4_launch(const Fp4Operand& x, const Fp4Operand& w, const float* b, const void* residual, void* y, int T,
                              int K, int N, int format, int act, int* status, cudaStream_t st) {
  Fp4Params p{};
  p.M = T;
  p.N = N;
  p.act = act;
  p.bias = b;
  p.scale_x = x.tensor_scale;
  p.scale_w = w.tensor_scale;
  p.status = status;
  const Fp4Tiling t = choose(T, N, K, format);
  // Few tokens as clusters where that is estimated shorter (clusters against tiles, codes of NVFP4: one token 6144 x 1536
  // 6.8 and 8.0 us, 8192 x 8192 10.6 and 18.9, 384 x 1152 4.4 and 3.2).
  if (T <= kFewTokens4) {
    const FewFp4Tiling few = few_fp4_tiling(T, N, K);
    if (few.cost < t.cost)
      return linear_fp4_few_launch(few, x.codes, x.scales, 1, x.tensor_scale, w, b, residual, y, T, K, N, format, act, status, st);
  }
  if (t.cg == 2)
    return format == 0 ? launch_tiles4<2, 0>(t.NT, x, w, residual, y, p, K, st)
                       : launch_tiles4<2, 1>(t.NT, x, w, residual, y, p, K, st);
  return format == 0 ? launch_tiles4<1, 0>(t.NT, x, w, residual, y, p, K, st)
                     : launch_tiles4<1, 1>(t.NT, x, w, residual, y, p, K, st);
}

}  // namespace swin
