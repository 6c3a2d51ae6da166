// C ABI of the swin_wattn library: argument validation, plan ownership, launches and
// error surfacing. No exception, abort or trap crosses this boundary.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <memory>
#include <mutex>
#include <new>
#include <unordered_set>
#include <vector>

#include "clip_grad.cuh"
#include "common.cuh"
#include "fp4.cuh"

namespace swin {
cudaError_t launch_bias_tables(const Plan& p, const float* table, bool with_mask, cudaStream_t st);
bool fwd_fp8_applies(const Plan& pl);
cudaError_t fwd_fp8_launch(const Plan& pl, const void* qkv8, float sq, float sk, float sv, void* out,
                           cudaStream_t st);
cudaError_t launch_build_mask(int H, int W, int M, int s, float* mask, cudaStream_t st);
cudaError_t launch_gather_map(int H, int W, int M, int s, int32_t* out, cudaStream_t st);
cudaError_t launch_relidx(int M, int32_t* out, cudaStream_t st);
size_t tc_tables_bytes(const Plan& pl);
cudaError_t launch_tc_tables(const Plan& pl, cudaStream_t st);
size_t bias_frag_bytes(int M, int nH);
size_t mask_frag_bytes(int M);
cudaError_t fwd_config(const Plan& pl, FwdLaunch* L);
cudaError_t fwd_launch(const Plan& pl, const FwdLaunch& L, const void* qkv, void* out,
                       cudaStream_t st);
cudaError_t fwd_launch_batch(const Plan& pl, const FwdLaunch& L, const void* qkv, void* out,
                             int batch, cudaStream_t st);
cudaError_t bwd_config(const Plan& pl, BwdLaunch* L);
bool bwd_tc_applies(const Plan& pl);
cudaError_t bwd_tc_config(const Plan& pl, BwdLaunch* L);
cudaError_t qkv_proj_launch(const void* x, const float* gamma, const float* beta, const void* w, const float* b,
                            void* out, int T, int C, float eps, void* workspace, int* status, cudaStream_t st);
size_t qkv_workspace_bytes(int C, int64_t T);
size_t qkv_prepared_bytes(int C);
size_t qkv_stats_bytes(int64_t T);
cudaError_t qkv_prepare_launch(const float* gamma, const float* beta, const void* w, const float* b, int C,
                               void* prepared, cudaStream_t st);
cudaError_t qkv_proj_prepared_launch(const void* x, const void* prepared, void* out, int T, int C, float eps,
                                     void* stats_workspace, int* status, cudaStream_t st);
int qkv_launches(int T, int C, bool fold);
cudaError_t qkv_proj_fp8_launch(const void* x, const void* prepared, void* out8, int T, int C, float eps,
                                const float scales[3], unsigned int* amax, void* stats_workspace, int* status,
                                cudaStream_t st);
cudaError_t proj_residual_launch(const void* o, const void* wp, const float* bp, const void* residual, void* y,
                                 int T, int C, int* status, cudaStream_t st);
cudaError_t bwd_launch(const Plan& pl, const BwdLaunch& L, const void* qkv, const void* dout,
                       void* dqkv, float* dtable, cudaStream_t st);
cudaError_t linear_launch(const void* x, const void* w, const float* b, const void* residual, void* y, void* pre,
                          int T, int K, int N, int act, int* status, cudaStream_t st);
cudaError_t linear_bwd_data_launch(const void* dy, const void* w, const void* pre, void* dx, int T, int K, int N,
                                   int act, int* status, cudaStream_t st);
size_t linear_bwd_weight_workspace_bytes(int64_t T, int K, int N);
int linear_bwd_weight_launches(int64_t T, int K, int N);
cudaError_t linear_bwd_weight_launch(const void* dy, const void* x, void* dw, float* db, int T, int K, int N,
                                     int dtype, int accumulate, void* workspace, int* status, cudaStream_t st);
size_t orthogonalize_workspace_bytes(int count, int rows, int cols);
int orthogonalize_launches(int count, int rows, int cols, int steps);
cudaError_t orthogonalize_launch(const void* g, void* out, int count, int rows, int cols, int dtype, int steps,
                                 float eps, float scale, void* workspace, int* status, cudaStream_t st);
cudaError_t block_norm_launch(const void* x, const void* f, const float* pre_w, const float* pre_b, const float* post_w,
                              const float* post_b, const float* gate, const float* keep, void* y, void* h, int tokens,
                              int C, int samples, int dtype, int kind, float alpha, float eps, cudaStream_t st);
size_t block_norm_bwd_workspace_bytes(int tokens, int C);
cudaError_t block_norm_bwd_launch(const void* y, const void* f, const void* dh, const void* dy, const float* pre_w,
                                  const float* post_w, const float* post_b, const float* gate, const float* keep,
                                  void* dx, void* df, float* dpre_w, float* dpre_b, float* dpost_w, float* dpost_b,
                                  float* dgate, int tokens, int C, int samples, int dtype, int kind, float alpha,
                                  float eps, int accumulate, void* workspace, cudaStream_t st);
size_t fp4_workspace_bytes();
cudaError_t fp4_quantize_launch(const void* x, void* codes, void* scales, float* tensor_scale, int rows, int K, int format,
                                int dtype, bool scale_given, void* workspace, cudaStream_t st);
cudaError_t fp4_dequantize_launch(const void* codes, const void* scales, const float* tensor_scale, void* out, int rows,
                                  int K, int format, int dtype, cudaStream_t st);
bool linear_fp4_quantizes(int T, int K, int N, int format);
cudaError_t linear_fp4_of_few(const void* x, int dtype, const float* x_scale, const Fp4Operand& w, const float* b,
                              const void* residual, void* y, int T, int K, int N, int format, int act, int* status,
                              cudaStream_t st);
cudaError_t linear_fp4_launch(const Fp4Operand& x, const Fp4Operand& w, const float* b, const void* residual, void* y, int T,
                              int K, int N, int format, int act, int* status, cudaStream_t st);
}  // namespace swin

// Streams and events of the host-buffer forward's copy/compute pipeline, created on
// its first use.
constexpr int kHostChunks = 4;
struct HostPipe {
  bool ready = false;
  cudaStream_t in = nullptr, out = nullptr;
  cudaEvent_t start = nullptr, done = nullptr;
  cudaEvent_t loaded[kHostChunks] = {}, computed[kHostChunks] = {};
};

struct swin_wattn_plan_s {
  swin::Plan p;
  swin::FwdLaunch fwd;
  swin::BwdLaunch bwd;
  HostPipe pipe;
};

// A plan of swin_wattn_clip_plan.
struct swin_wattn_clip_s {
  swin::ClipShape shape;
  const swin::ClipPiece* list;  // device memory, the caller's
  std::vector<std::pair<uint64_t, uint64_t>> spans;  // of all its bytes, joined and in order
  int device;
};

namespace {

thread_local char g_last_error[256] = "";
thread_local uint64_t g_launches = 0;

int cuda_fail(cudaError_t e, const char* where) {
  std::snprintf(g_last_error, sizeof(g_last_error), "%s: %s (%s)", where, cudaGetErrorName(e),
                cudaGetErrorString(e));
  return SWIN_WATTN_ERR_CUDA;
}

// A pointer the GPU can dereference: device or managed memory, or host memory mapped
// into the device address space.
int check_device_ptr(const void* ptr, size_t align) {
  if (ptr == nullptr) return SWIN_WATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ptr) % align != 0) return SWIN_WATTN_ERR_MISALIGNED;
  cudaPointerAttributes a;
  cudaError_t e = cudaPointerGetAttributes(&a, ptr);
  if (e != cudaSuccess) {
    cudaGetLastError();  // clear the sticky-free error state of this query
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  if (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged) return SWIN_WATTN_OK;
  if (a.type == cudaMemoryTypeHost && a.devicePointer == ptr) return SWIN_WATTN_OK;
  return SWIN_WATTN_ERR_INVALID_ARG;
}

// A device pointer, as above, of memory that lies on device `dev` (or is mapped).
int check_on_device(const void* ptr, size_t align, int dev) {
  if (reinterpret_cast<uintptr_t>(ptr) % align != 0) return SWIN_WATTN_ERR_MISALIGNED;
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
    cudaGetLastError();
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  if (a.type == cudaMemoryTypeDevice) return a.device == dev ? SWIN_WATTN_OK : SWIN_WATTN_ERR_INVALID_ARG;
  if (a.type == cudaMemoryTypeManaged) return SWIN_WATTN_OK;
  return a.type == cudaMemoryTypeHost && a.devicePointer == ptr ? SWIN_WATTN_OK : SWIN_WATTN_ERR_INVALID_ARG;
}

// A buffer of a call: its pointer, size and alignment.
struct Buffer {
  const void* ptr;
  uint64_t bytes;
  size_t align;
  bool written;
};

bool overlaps(const Buffer& a, const Buffer& b) {
  const uint64_t pa = reinterpret_cast<uintptr_t>(a.ptr), pb = reinterpret_cast<uintptr_t>(b.ptr);
  return pa < pb + b.bytes && pb < pa + a.bytes;
}

// Every buffer that is given is memory of the current device, and none that is written
// overlaps another, except buffer `same_a` that is buffer `same_b` itself.
int check_buffers(const char* where, const Buffer* bufs, int n, int same_a = -1, int same_b = -1) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; ++i) {
    if (bufs[i].ptr == nullptr) continue;
    const int rc = check_on_device(bufs[i].ptr, bufs[i].align, dev);
    if (rc != SWIN_WATTN_OK) return rc;
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if (bufs[i].ptr == nullptr || bufs[j].ptr == nullptr || !(bufs[i].written || bufs[j].written)) continue;
      if (i == same_a && j == same_b && bufs[i].ptr == bufs[j].ptr) continue;
      if (overlaps(bufs[i], bufs[j])) {
        std::snprintf(g_last_error, sizeof(g_last_error), "%s: overlapping buffers", where);
        return SWIN_WATTN_ERR_INVALID_ARG;
      }
    }
  return SWIN_WATTN_OK;
}

// Tile rows past the last token still have to fit an int.
constexpr int kMaxLinearTokens = 0x7fffffff - 1023;
bool linear_width(int n) { return n >= 8 && n <= 32768 && n % 8 == 0; }
bool known_act(int act) { return act >= SWIN_WATTN_ACT_NONE && act <= SWIN_WATTN_ACT_SILU; }

// Live plans. A handle is checked against this set before it is dereferenced, so a
// destroyed or foreign handle is reported instead of read.
std::mutex g_plans_mu;
std::unordered_set<const swin_wattn_plan_s*> g_plans;

int check_plan(const swin_wattn_plan_s* pl) {
  if (pl == nullptr) return SWIN_WATTN_ERR_BAD_PLAN;
  {
    std::lock_guard<std::mutex> lk(g_plans_mu);
    if (g_plans.find(pl) == g_plans.end()) return SWIN_WATTN_ERR_BAD_PLAN;
  }
  if (pl->p.magic != swin::kPlanMagic) return SWIN_WATTN_ERR_BAD_PLAN;
  return SWIN_WATTN_OK;
}

std::unordered_set<const swin_wattn_clip_s*> g_clips;  // under g_plans_mu

int check_clip(const swin_wattn_clip_s* pl) {
  std::lock_guard<std::mutex> lk(g_plans_mu);
  return pl != nullptr && g_clips.find(pl) != g_clips.end() ? SWIN_WATTN_OK : SWIN_WATTN_ERR_BAD_PLAN;
}

bool normal_eps(float eps) { return eps >= FLT_MIN && std::isfinite(eps); }
bool float_dtype(int dtype) { return dtype == SWIN_WATTN_FP32 || dtype == SWIN_WATTN_BF16; }
bool norm_width(int C) { return C >= 8 && C <= 8192 && C % 8 == 0; }
bool fp4_width(int K) { return K >= 32 && K <= 32768 && K % 32 == 0; }
bool fp4_format(int f) { return f == SWIN_WATTN_NVFP4 || f == SWIN_WATTN_MXFP4; }

void free_pipe(HostPipe& hp) {
  if (!hp.ready) return;
  for (int c = 0; c < kHostChunks; ++c) {
    cudaEventDestroy(hp.loaded[c]);
    cudaEventDestroy(hp.computed[c]);
  }
  cudaEventDestroy(hp.start);
  cudaEventDestroy(hp.done);
  cudaStreamDestroy(hp.in);
  cudaStreamDestroy(hp.out);
  hp.ready = false;
}

void free_plan_buffers(swin::Plan& p) {
  if (p.dense_bias) cudaFree(p.dense_bias);
  if (p.mask) cudaFree(p.mask);
  if (p.dt_partial) cudaFree(p.dt_partial);
  if (p.bias_frag) cudaFree(p.bias_frag);
  if (p.mask_frag) cudaFree(p.mask_frag);
  if (p.err) cudaFree(p.err);
  if (p.tc_tables) cudaFree(p.tc_tables);

  p.dense_bias = p.mask = p.dt_partial = nullptr;
  p.bias_frag = nullptr;
  p.mask_frag = nullptr;
  p.err = nullptr;
  p.tc_tables = nullptr;
}

}  // namespace

namespace swin {
void set_last_error(const char* msg) { std::snprintf(g_last_error, sizeof(g_last_error), "%s", msg); }
int check_device_ptr_abi(const void* ptr, size_t align) { return check_device_ptr(ptr, align); }
// Kernel launches issued by the calling thread outside this file (swin_wattn_launch_count).
void count_launches(int n) { g_launches += (uint64_t)n; }

namespace {
std::atomic<uint64_t> g_wait_ns{1000000000ull};
std::atomic<int> g_fault{kFaultNone};
}  // namespace
uint64_t wait_limit_ns() { return g_wait_ns.load(std::memory_order_relaxed); }
int fault_site() { return g_fault.load(std::memory_order_relaxed); }
}  // namespace swin

#ifdef SWIN_WATTN_FAULT_INJECTION
#include "../../include/swin_wattn_debug.h"

extern "C" int swin_wattn_debug_set_fault(int site, int64_t wait_limit_ns) {
  if (site < swin::kFaultNone || site > swin::kFaultGemm) return SWIN_WATTN_ERR_INVALID_ARG;
  if (wait_limit_ns < 1000 || wait_limit_ns > 10000000000ll) return SWIN_WATTN_ERR_INVALID_ARG;
  swin::g_wait_ns.store((uint64_t)wait_limit_ns);
  swin::g_fault.store(site);
  return SWIN_WATTN_OK;
}
#endif

extern "C" {

const char* swin_wattn_status_string(int status) {
  switch (status) {
    case SWIN_WATTN_OK: return "ok";
    case SWIN_WATTN_ERR_INVALID_ARG: return "invalid argument";
    case SWIN_WATTN_ERR_UNSUPPORTED: return "unsupported shape";
    case SWIN_WATTN_ERR_MISALIGNED: return "misaligned pointer";
    case SWIN_WATTN_ERR_BAD_PLAN: return "bad plan handle";
    case SWIN_WATTN_ERR_CUDA: return "CUDA error";
    case SWIN_WATTN_ERR_TIMEOUT: return "device wait timed out";
    default: return "unknown status";
  }
}

const char* swin_wattn_last_error(void) { return g_last_error; }

uint64_t swin_wattn_launch_count(int reset) {
  const uint64_t n = g_launches;
  if (reset) g_launches = 0;
  return n;
}

int swin_wattn_plan(swin_wattn_plan_t* out, int B, int H, int W, int C, int num_heads,
                    int window, int shift, int dtype, const float* bias_table,
                    struct CUstream_st* stream) {
  if (out == nullptr) return SWIN_WATTN_ERR_INVALID_ARG;
  *out = nullptr;
  if (B < 0 || H <= 0 || W <= 0 || C <= 0 || num_heads <= 0) return SWIN_WATTN_ERR_INVALID_ARG;
  if (dtype != SWIN_WATTN_BF16 && dtype != SWIN_WATTN_FP32) return SWIN_WATTN_ERR_INVALID_ARG;
  if (window != 4 && window != 7 && window != 12) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (shift < 0 || shift >= window) return SWIN_WATTN_ERR_INVALID_ARG;
  if (H % window != 0 || W % window != 0) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (C % num_heads != 0 || C / num_heads != swin::kHeadDim) return SWIN_WATTN_ERR_UNSUPPORTED;
  if ((int64_t)B * H * W * 3 * C >= ((int64_t)1 << 40)) return SWIN_WATTN_ERR_UNSUPPORTED;
  int rc = check_device_ptr(bias_table, 4);
  if (rc != SWIN_WATTN_OK) return rc;

  swin_wattn_plan_s* pl = new (std::nothrow) swin_wattn_plan_s();
  if (pl == nullptr) return SWIN_WATTN_ERR_INVALID_ARG;
  swin::Plan& p = pl->p;
  std::memset(&p, 0, sizeof(p));
  p.B = B;
  p.H = H;
  p.W = W;
  p.C = C;
  p.nH = num_heads;
  p.M = window;
  p.s = shift;
  p.dtype = dtype;
  p.N = window * window;
  p.nWy = H / window;
  p.nWx = W / window;
  p.nW = p.nWy * p.nWx;

  cudaError_t e = cudaGetDevice(&p.device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&p.num_sms, cudaDevAttrMultiProcessorCount, p.device);
  const size_t nn = (size_t)p.N * p.N;
  if (e == cudaSuccess) e = cudaMalloc(&p.dense_bias, sizeof(float) * nn * p.nH);
  // The mask tensor always exists (all zeros for s = 0) so that it can be dumped.
  if (e == cudaSuccess) e = cudaMalloc(&p.mask, sizeof(float) * nn * p.nW);
  if (e == cudaSuccess) e = cudaMalloc(&p.bias_frag, swin::bias_frag_bytes(p.M, p.nH));
  if (e == cudaSuccess && p.s > 0) e = cudaMalloc(&p.mask_frag, swin::mask_frag_bytes(p.M));
  if (e == cudaSuccess) e = cudaMalloc(&p.err, sizeof(int));
  if (e == cudaSuccess && swin::tc_tables_bytes(p) > 0) e = cudaMalloc(&p.tc_tables, swin::tc_tables_bytes(p));
  if (e == cudaSuccess) e = cudaMemsetAsync(p.err, 0, sizeof(int), reinterpret_cast<cudaStream_t>(stream));

  if (e == cudaSuccess) e = swin::fwd_config(p, &pl->fwd);
  if (e == cudaSuccess) e = swin::bwd_config(p, &pl->bwd);
  // the table-gradient partials, sized for either backward kernel (the choice may change)
  int partial_rows = pl->bwd.partial_rows;
  if (e == cudaSuccess && swin::bwd_tc_applies(p)) {
    swin::BwdLaunch Lt;
    e = swin::bwd_tc_config(p, &Lt);
    if (e == cudaSuccess && Lt.partial_rows > partial_rows) partial_rows = Lt.partial_rows;
  }
  if (e == cudaSuccess && partial_rows > 0) {
    p.dt_partial_rows = partial_rows;
    e = cudaMalloc(&p.dt_partial, sizeof(float) * (size_t)p.dt_partial_rows * (2 * p.M - 1) *
                                      (2 * p.M - 1));
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (e == cudaSuccess) {
    e = swin::launch_bias_tables(p, bias_table, true, st);
    ++g_launches;
  }
  if (e == cudaSuccess) {
    e = swin::launch_build_mask(p.H, p.W, p.M, p.s, p.mask, st);
    ++g_launches;
  }
  p.tc_stale = p.tc_tables != nullptr;  // built before the first tcgen05 forward
  if (e != cudaSuccess) {
    rc = cuda_fail(e, "swin_wattn_plan");
    free_plan_buffers(p);
    delete pl;
    return rc;
  }
  p.magic = swin::kPlanMagic;
  {
    std::lock_guard<std::mutex> lk(g_plans_mu);
    g_plans.insert(pl);
  }
  *out = pl;
  return SWIN_WATTN_OK;
}

int swin_wattn_set_bias(swin_wattn_plan_t plan, const float* bias_table,
                        struct CUstream_st* stream) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  rc = check_device_ptr(bias_table, 4);
  if (rc != SWIN_WATTN_OK) return rc;
  swin::Plan& p = plan->p;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // One launch: the mma fragments and the dense bias, both from the table. The tcgen05
  // tables are rebuilt before the next forward that uses them.
  cudaError_t e = swin::launch_bias_tables(p, bias_table, false, st);
  ++g_launches;
  p.tc_stale = p.tc_tables != nullptr;
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_set_bias");
}

// The tcgen05 forward's constant tables, rebuilt from the dense bias on `st` when the bias
// changed since they were last built.
static cudaError_t ensure_tc_tables(swin_wattn_plan_s* plan, cudaStream_t st, bool for_bwd = false) {
  swin::Plan& p = plan->p;
  if (!(for_bwd ? plan->bwd.tc : plan->fwd.tc) || !p.tc_stale) return cudaSuccess;
  const cudaError_t e = swin::launch_tc_tables(p, st);
  ++g_launches;
  if (e == cudaSuccess) p.tc_stale = false;
  return e;
}

int swin_wattn_fwd(swin_wattn_plan_t plan, const void* qkv, void* out,
                   struct CUstream_st* stream) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  const swin::Plan& p = plan->p;
  if (p.B == 0) return SWIN_WATTN_OK;
  if ((rc = check_device_ptr(qkv, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(out, 16)) != SWIN_WATTN_OK) return rc;
  cudaError_t e = ensure_tc_tables(plan, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = swin::fwd_launch(p, plan->fwd, qkv, out, reinterpret_cast<cudaStream_t>(stream));
  ++g_launches;
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_fwd");
}

int swin_wattn_fwd_fp8(swin_wattn_plan_t plan, const void* qkv8, float scale_q, float scale_k, float scale_v,
                       void* out, struct CUstream_st* stream) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  const swin::Plan& p = plan->p;
  if (!swin::fwd_fp8_applies(p)) return SWIN_WATTN_ERR_UNSUPPORTED;
  for (const float sc : {scale_q, scale_k, scale_v})
    if (!(sc > 0.0f) || !std::isfinite(sc)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale_q * scale_k) || !(scale_q * scale_k > 0.0f)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (p.B == 0) return SWIN_WATTN_OK;
  if ((rc = check_device_ptr(qkv8, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(out, 16)) != SWIN_WATTN_OK) return rc;
  cudaError_t e = swin::fwd_fp8_launch(p, qkv8, scale_q, scale_k, scale_v, out, reinterpret_cast<cudaStream_t>(stream));
  ++g_launches;
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_fwd_fp8");
}

int swin_wattn_fwd_host(swin_wattn_plan_t plan, const void* qkv_host, void* out_host,
                        void* dev_qkv, void* dev_out, struct CUstream_st* stream) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  const swin::Plan& p = plan->p;
  if (p.B == 0) return SWIN_WATTN_OK;
  if (qkv_host == nullptr || out_host == nullptr) return SWIN_WATTN_ERR_INVALID_ARG;
  if ((rc = check_device_ptr(dev_qkv, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(dev_out, 16)) != SWIN_WATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = ensure_tc_tables(plan, st);
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_fwd_host");
  HostPipe& hp = plan->pipe;
  if (!hp.ready) {
    e = cudaStreamCreateWithFlags(&hp.in, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&hp.out, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&hp.start, cudaEventDisableTiming);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&hp.done, cudaEventDisableTiming);
    for (int c = 0; c < kHostChunks && e == cudaSuccess; ++c) {
      e = cudaEventCreateWithFlags(&hp.loaded[c], cudaEventDisableTiming);
      if (e == cudaSuccess) e = cudaEventCreateWithFlags(&hp.computed[c], cudaEventDisableTiming);
    }
    if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_fwd_host");
    hp.ready = true;
  }
  // Batch chunks flow through three queues: copy-in, compute (the caller's stream) and
  // copy-out, so the two copy directions and the kernels overlap; the caller's stream
  // finally waits for the last copy-out, keeping the call ordered on `stream`.
  const size_t esz = p.dtype == SWIN_WATTN_FP32 ? 4 : 2;
  const size_t img_in = (size_t)p.H * p.W * 3 * p.C * esz, img_out = (size_t)p.H * p.W * p.C * esz;
  const int nchunk = p.B < kHostChunks ? p.B : kHostChunks;
  e = cudaEventRecord(hp.start, st);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(hp.in, hp.start, 0);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(hp.out, hp.start, 0);
  for (int c = 0; c < nchunk && e == cudaSuccess; ++c) {
    const int b0 = (int)((int64_t)p.B * c / nchunk), b1 = (int)((int64_t)p.B * (c + 1) / nchunk);
    const size_t n_in = img_in * (b1 - b0), n_out = img_out * (b1 - b0);
    const char* hsrc = static_cast<const char*>(qkv_host) + img_in * b0;
    char* dq = static_cast<char*>(dev_qkv) + img_in * b0;
    char* dout = static_cast<char*>(dev_out) + img_out * b0;
    e = cudaMemcpyAsync(dq, hsrc, n_in, cudaMemcpyHostToDevice, hp.in);
    if (e == cudaSuccess) e = cudaEventRecord(hp.loaded[c], hp.in);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(st, hp.loaded[c], 0);
    if (e == cudaSuccess) {
      e = swin::fwd_launch_batch(p, plan->fwd, dq, dout, b1 - b0, st);
      ++g_launches;
    }
    if (e == cudaSuccess) e = cudaEventRecord(hp.computed[c], st);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(hp.out, hp.computed[c], 0);
    if (e == cudaSuccess)
      e = cudaMemcpyAsync(static_cast<char*>(out_host) + img_out * b0, dout, n_out,
                          cudaMemcpyDeviceToHost, hp.out);
  }
  if (e == cudaSuccess) e = cudaEventRecord(hp.done, hp.out);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(st, hp.done, 0);
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_fwd_host");
}

int swin_wattn_bwd(swin_wattn_plan_t plan, const void* qkv, const void* dout, void* dqkv,
                   float* dtable, struct CUstream_st* stream) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  const swin::Plan& p = plan->p;
  if (plan->bwd.grid == 0 && p.B > 0) return SWIN_WATTN_ERR_UNSUPPORTED;
  if ((rc = check_device_ptr(dtable, 4)) != SWIN_WATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t tbytes = sizeof(float) * (size_t)(2 * p.M - 1) * (2 * p.M - 1) * p.nH;
  if (p.B == 0) {
    cudaError_t e = cudaMemsetAsync(dtable, 0, tbytes, st);
    return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_bwd");
  }
  if ((rc = check_device_ptr(qkv, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(dout, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(dqkv, 16)) != SWIN_WATTN_OK) return rc;
  cudaError_t e = ensure_tc_tables(plan, st, true);
  if (e == cudaSuccess) e = swin::bwd_launch(p, plan->bwd, qkv, dout, dqkv, dtable, st);
  g_launches += 2;
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_bwd");
}

int swin_wattn_debug_maps(swin_wattn_plan_t plan, int32_t* gather, int32_t* relidx,
                          float* mask, float* dense_bias, struct CUstream_st* stream) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  const swin::Plan& p = plan->p;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t nn = (size_t)p.N * p.N;
  cudaError_t e = cudaSuccess;
  if (gather) {
    if ((rc = check_device_ptr(gather, 4)) != SWIN_WATTN_OK) return rc;
    e = swin::launch_gather_map(p.H, p.W, p.M, p.s, gather, st);
    ++g_launches;
  }
  if (e == cudaSuccess && relidx) {
    if ((rc = check_device_ptr(relidx, 4)) != SWIN_WATTN_OK) return rc;
    e = swin::launch_relidx(p.M, relidx, st);
    ++g_launches;
  }
  if (e == cudaSuccess && mask) {
    if ((rc = check_device_ptr(mask, 4)) != SWIN_WATTN_OK) return rc;
    e = cudaMemcpyAsync(mask, p.mask, sizeof(float) * nn * p.nW, cudaMemcpyDeviceToDevice, st);
  }
  if (e == cudaSuccess && dense_bias) {
    if ((rc = check_device_ptr(dense_bias, 4)) != SWIN_WATTN_OK) return rc;
    e = cudaMemcpyAsync(dense_bias, p.dense_bias, sizeof(float) * nn * p.nH,
                        cudaMemcpyDeviceToDevice, st);
  }
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_debug_maps");
}

size_t swin_wattn_qkv_workspace_bytes(int C, int tokens) {
  return (C < 32 || C > 1536 || C % 32 != 0 || tokens < 0) ? 0 : swin::qkv_workspace_bytes(C, tokens);
}

int swin_wattn_qkv_proj(const void* x, const float* gamma, const float* beta, const void* w_qkv,
                        const float* b_qkv, void* qkv, int tokens, int C, float eps, void* workspace,
                        size_t workspace_bytes, int* status, struct CUstream_st* stream) {
  if (tokens < 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (C < 32 || C > 1536 || C % 32 != 0) return SWIN_WATTN_ERR_UNSUPPORTED;
  if ((int64_t)tokens >= ((int64_t)1 << 31)) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return SWIN_WATTN_OK;
  if (workspace_bytes < swin::qkv_workspace_bytes(C, tokens)) {
    swin::set_last_error("swin_wattn_qkv_proj: workspace smaller than swin_wattn_qkv_workspace_bytes(C, tokens)");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  int rc;
  if ((rc = check_device_ptr(x, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(w_qkv, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(qkv, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(workspace, 256)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(gamma, 4)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(beta, 4)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(b_qkv, 4)) != SWIN_WATTN_OK) return rc;
  if (status != nullptr && (rc = check_device_ptr(status, 4)) != SWIN_WATTN_OK) return rc;
  cudaError_t e = swin::qkv_proj_launch(x, gamma, beta, w_qkv, b_qkv, qkv, tokens, C, eps, workspace, status,
                                        reinterpret_cast<cudaStream_t>(stream));
  g_launches += 2;
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_qkv_proj");
}

size_t swin_wattn_qkv_prepared_bytes(int C) {
  return (C < 32 || C > 1536 || C % 32 != 0) ? 0 : swin::qkv_prepared_bytes(C);
}

size_t swin_wattn_qkv_stats_bytes(int tokens) { return tokens < 0 ? 0 : swin::qkv_stats_bytes(tokens); }

int swin_wattn_qkv_prepare(const float* gamma, const float* beta, const void* w_qkv, const float* b_qkv, int C,
                           void* prepared, size_t prepared_bytes, struct CUstream_st* stream) {
  if (C < 32 || C > 1536 || C % 32 != 0) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (prepared_bytes < swin::qkv_prepared_bytes(C)) {
    swin::set_last_error("swin_wattn_qkv_prepare: buffer smaller than swin_wattn_qkv_prepared_bytes(C)");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  int rc;
  if ((rc = check_device_ptr(w_qkv, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(prepared, 256)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(gamma, 4)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(beta, 4)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(b_qkv, 4)) != SWIN_WATTN_OK) return rc;
  cudaError_t e = swin::qkv_prepare_launch(gamma, beta, w_qkv, b_qkv, C, prepared,
                                           reinterpret_cast<cudaStream_t>(stream));
  ++g_launches;
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_qkv_prepare");
}

int swin_wattn_qkv_proj_prepared(const void* x, const void* prepared, void* qkv, int tokens, int C, float eps,
                                 void* stats_workspace, size_t stats_bytes, int* status, struct CUstream_st* stream) {
  if (tokens < 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (C < 32 || C > 1536 || C % 32 != 0) return SWIN_WATTN_ERR_UNSUPPORTED;
  if ((int64_t)tokens >= ((int64_t)1 << 31)) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return SWIN_WATTN_OK;
  if (stats_bytes < swin::qkv_stats_bytes(tokens)) {
    swin::set_last_error("swin_wattn_qkv_proj_prepared: statistics workspace smaller than "
                         "swin_wattn_qkv_stats_bytes(tokens)");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  int rc;
  if ((rc = check_device_ptr(x, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(prepared, 256)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(qkv, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(stats_workspace, 16)) != SWIN_WATTN_OK) return rc;
  if (status != nullptr && (rc = check_device_ptr(status, 4)) != SWIN_WATTN_OK) return rc;
  cudaError_t e = swin::qkv_proj_prepared_launch(x, prepared, qkv, tokens, C, eps, stats_workspace, status,
                                                 reinterpret_cast<cudaStream_t>(stream));
  g_launches += swin::qkv_launches(tokens, C, false);
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_qkv_proj_prepared");
}

int swin_wattn_qkv_proj_prepared_fp8(const void* x, const void* prepared, void* qkv8, int tokens, int C, float eps,
                                     float scale_q, float scale_k, float scale_v, float* amax, void* stats_workspace,
                                     size_t stats_bytes, int* status, struct CUstream_st* stream) {
  if (tokens < 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return SWIN_WATTN_ERR_INVALID_ARG;
  for (const float sc : {scale_q, scale_k, scale_v})
    if (!(sc > 0.0f) || !std::isfinite(sc) || !std::isfinite(1.0f / sc)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (C < 32 || C > 1536 || C % 32 != 0) return SWIN_WATTN_ERR_UNSUPPORTED;
  if ((int64_t)tokens >= ((int64_t)1 << 31)) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return SWIN_WATTN_OK;
  if (stats_bytes < swin::qkv_stats_bytes(tokens)) {
    swin::set_last_error("swin_wattn_qkv_proj_prepared_fp8: statistics workspace smaller than "
                         "swin_wattn_qkv_stats_bytes(tokens)");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  int rc;
  if ((rc = check_device_ptr(x, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(prepared, 256)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(qkv8, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(stats_workspace, 16)) != SWIN_WATTN_OK) return rc;
  if (amax != nullptr && (rc = check_device_ptr(amax, 4)) != SWIN_WATTN_OK) return rc;
  if (status != nullptr && (rc = check_device_ptr(status, 4)) != SWIN_WATTN_OK) return rc;
  const float scales[3] = {scale_q, scale_k, scale_v};
  cudaError_t e = swin::qkv_proj_fp8_launch(x, prepared, qkv8, tokens, C, eps, scales,
                                            reinterpret_cast<unsigned int*>(amax), stats_workspace, status,
                                            reinterpret_cast<cudaStream_t>(stream));
  g_launches += swin::qkv_launches(tokens, C, false);
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_qkv_proj_prepared_fp8");
}

int swin_wattn_proj_residual(const void* o, const void* w_proj, const float* b_proj, const void* residual,
                             void* y, int tokens, int C, int* status, struct CUstream_st* stream) {
  if (tokens < 0) return SWIN_WATTN_ERR_INVALID_ARG;
  if (C < 32 || C > 1536 || C % 32 != 0) return SWIN_WATTN_ERR_UNSUPPORTED;
  if ((int64_t)tokens >= ((int64_t)1 << 31)) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return SWIN_WATTN_OK;
  int rc;
  if ((rc = check_device_ptr(o, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(w_proj, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(residual, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(y, 16)) != SWIN_WATTN_OK) return rc;
  if ((rc = check_device_ptr(b_proj, 4)) != SWIN_WATTN_OK) return rc;
  if (status != nullptr && (rc = check_device_ptr(status, 4)) != SWIN_WATTN_OK) return rc;
  const uintptr_t ob = reinterpret_cast<uintptr_t>(o), yb = reinterpret_cast<uintptr_t>(y);
  const uintptr_t bytes = (uintptr_t)tokens * (uintptr_t)C * 2;
  if (ob < yb + bytes && yb < ob + bytes) {
    swin::set_last_error("swin_wattn_proj_residual: y overlaps o");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  cudaError_t e = swin::proj_residual_launch(o, w_proj, b_proj, residual, y, tokens, C, status,
                                             reinterpret_cast<cudaStream_t>(stream));
  ++g_launches;
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_proj_residual");
}

int swin_wattn_linear(const void* x, const void* w, const float* b, const void* residual, void* y, void* pre,
                      int tokens, int K, int N, int act, int* status, struct CUstream_st* stream) {
  if (tokens < 0 || !known_act(act)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (!linear_width(K) || !linear_width(N) || tokens > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return SWIN_WATTN_OK;
  if (x == nullptr || w == nullptr || y == nullptr) return SWIN_WATTN_ERR_INVALID_ARG;
  const uint64_t T = (uint64_t)tokens;
  const Buffer bufs[] = {{x, T * K * 2, 16, false}, {w, (uint64_t)N * K * 2, 16, false}, {b, (uint64_t)N * 4, 4, false},
                         {residual, T * N * 2, 16, false}, {y, T * N * 2, 16, true}, {pre, T * N * 2, 16, true},
                         {status, 4, 4, true}};
  int rc = check_buffers("swin_wattn_linear", bufs, 7, 3, 4);
  if (rc != SWIN_WATTN_OK) return rc;
  cudaError_t e = swin::linear_launch(x, w, b, residual, y, pre, tokens, K, N, act, status,
                                      reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_linear");
  ++g_launches;
  return SWIN_WATTN_OK;
}

int swin_wattn_linear_bwd_data(const void* dy, const void* w, const void* pre, void* dx, int tokens, int K, int N,
                               int act, int* status, struct CUstream_st* stream) {
  if (tokens < 0 || !known_act(act)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (!linear_width(K) || !linear_width(N) || tokens > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return SWIN_WATTN_OK;
  if (act == SWIN_WATTN_ACT_NONE) pre = nullptr;
  if (dy == nullptr || w == nullptr || dx == nullptr || (act != SWIN_WATTN_ACT_NONE && pre == nullptr))
    return SWIN_WATTN_ERR_INVALID_ARG;
  const uint64_t T = (uint64_t)tokens;
  const Buffer bufs[] = {{dy, T * N * 2, 16, false}, {w, (uint64_t)N * K * 2, 16, false}, {pre, T * K * 2, 16, false},
                         {dx, T * K * 2, 16, true}, {status, 4, 4, true}};
  int rc = check_buffers("swin_wattn_linear_bwd_data", bufs, 5, 2, 3);
  if (rc != SWIN_WATTN_OK) return rc;
  cudaError_t e = swin::linear_bwd_data_launch(dy, w, pre, dx, tokens, K, N, act, status,
                                               reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_linear_bwd_data");
  ++g_launches;
  return SWIN_WATTN_OK;
}

size_t swin_wattn_linear_bwd_weight_workspace_bytes(int tokens, int K, int N) {
  if (tokens < 0 || tokens > kMaxLinearTokens || !linear_width(K) || !linear_width(N)) return 0;
  return swin::linear_bwd_weight_workspace_bytes(tokens, K, N);
}

int swin_wattn_linear_bwd_weight(const void* dy, const void* x, void* dw, float* db, int tokens, int K, int N,
                                 int dtype, int accumulate, void* workspace, size_t workspace_bytes, int* status,
                                 struct CUstream_st* stream) {
  if (tokens < 0 || (dtype != SWIN_WATTN_FP32 && dtype != SWIN_WATTN_BF16)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (!linear_width(K) || !linear_width(N) || tokens > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (dw == nullptr || (tokens > 0 && (dy == nullptr || x == nullptr || workspace == nullptr)))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (tokens > 0 && workspace_bytes < swin::linear_bwd_weight_workspace_bytes(tokens, K, N)) {
    swin::set_last_error("swin_wattn_linear_bwd_weight: workspace smaller than "
                         "swin_wattn_linear_bwd_weight_workspace_bytes(tokens, K, N)");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  const uint64_t T = (uint64_t)tokens;
  const Buffer bufs[] = {{T ? dy : nullptr, T * N * 2, 16, false}, {T ? x : nullptr, T * K * 2, 16, false},
                         {dw, (uint64_t)N * K * (dtype == SWIN_WATTN_FP32 ? 4 : 2), 16, true},
                         {db, (uint64_t)N * 4, 4, true}, {T ? workspace : nullptr, workspace_bytes, 256, true},
                         {status, 4, 4, true}};
  int rc = check_buffers("swin_wattn_linear_bwd_weight", bufs, 6);
  if (rc != SWIN_WATTN_OK) return rc;
  cudaError_t e = swin::linear_bwd_weight_launch(dy, x, dw, db, tokens, K, N, dtype, accumulate, workspace, status,
                                                 reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_linear_bwd_weight");
  g_launches += swin::linear_bwd_weight_launches(tokens, K, N);
  return SWIN_WATTN_OK;
}

static bool orthogonalize_sizes(int count, int rows, int cols) {
  return count >= 0 && count <= 65535 && rows >= 1 && rows <= 16384 && cols >= 1 && cols <= 16384;
}

size_t swin_wattn_orthogonalize_workspace_bytes(int count, int rows, int cols) {
  return orthogonalize_sizes(count, rows, cols) ? swin::orthogonalize_workspace_bytes(count, rows, cols) : 0;
}

int swin_wattn_orthogonalize(const void* g, void* out, int count, int rows, int cols, int dtype, int steps, float eps,
                             float scale, void* workspace, size_t workspace_bytes, int* status,
                             struct CUstream_st* stream) {
  if (count < 0 || (dtype != SWIN_WATTN_FP32 && dtype != SWIN_WATTN_BF16)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (!(eps >= FLT_MIN) || !std::isfinite(eps) || !std::isfinite(scale) || steps < 1 || steps > 20)
    return SWIN_WATTN_ERR_INVALID_ARG;
  // (the last product's factor, scale / 2^16 times a gain, stays a normal number)
  if (scale != 0.0f && std::fabs(scale) < 0x1p-100f) return SWIN_WATTN_ERR_INVALID_ARG;
  if (!orthogonalize_sizes(count, rows, cols)) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (count == 0) return SWIN_WATTN_OK;
  if (g == nullptr || out == nullptr || workspace == nullptr) return SWIN_WATTN_ERR_INVALID_ARG;
  if (workspace_bytes < swin::orthogonalize_workspace_bytes(count, rows, cols)) {
    swin::set_last_error("swin_wattn_orthogonalize: workspace smaller than "
                         "swin_wattn_orthogonalize_workspace_bytes(count, rows, cols)");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  const uint64_t elements = (uint64_t)count * rows * cols;
  const size_t elem = dtype == SWIN_WATTN_FP32 ? 4 : 2;
  const Buffer bufs[] = {{g, elements * elem, elem, false}, {out, elements * 2, 2, true},
                         {workspace, workspace_bytes, 256, true}, {status, 4, 4, true}};
  int rc = check_buffers("swin_wattn_orthogonalize", bufs, 4);
  if (rc != SWIN_WATTN_OK) return rc;
  cudaError_t e = swin::orthogonalize_launch(g, out, count, rows, cols, dtype, steps, eps, scale, workspace, status,
                                             reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_orthogonalize");
  g_launches += swin::orthogonalize_launches(count, rows, cols, steps);
  return SWIN_WATTN_OK;
}

int swin_wattn_block_norm(const void* x, const void* f, const float* pre_w, const float* pre_b, const float* post_w,
                          const float* post_b, const float* gate, const float* keep, void* y, void* h, int tokens, int C,
                          int samples, int dtype, int kind, float alpha, float eps, struct CUstream_st* stream) {
  if (tokens < 0 || !float_dtype(dtype) || (kind != SWIN_WATTN_NORM_LAYER && kind != SWIN_WATTN_NORM_RMS) ||
      !normal_eps(eps) || !std::isfinite(alpha))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (!norm_width(C) || tokens > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (keep != nullptr && (samples < 1 || tokens % samples != 0)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (tokens == 0) return SWIN_WATTN_OK;  // (tensors of no elements have no address to tell them by)
  if (f == nullptr ? post_w != nullptr || gate != nullptr || keep != nullptr || y != nullptr || pre_w == nullptr : y == nullptr)
    return SWIN_WATTN_ERR_INVALID_ARG;
  if ((pre_w == nullptr && (pre_b != nullptr || h != nullptr)) || (post_w == nullptr && post_b != nullptr))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (x == nullptr || (pre_w != nullptr && h == nullptr)) return SWIN_WATTN_ERR_INVALID_ARG;
  const uint64_t n = (uint64_t)tokens * C, stream_bytes = n * (dtype == SWIN_WATTN_FP32 ? 4 : 2), c4 = (uint64_t)C * 4;
  const Buffer bufs[] = {{x, stream_bytes, 16, false}, {y, stream_bytes, 16, true}, {f, n * 2, 16, false},
                         {h, n * 2, 16, true}, {pre_w, c4, 4, false}, {pre_b, c4, 4, false}, {post_w, c4, 4, false},
                         {post_b, c4, 4, false}, {gate, c4, 4, false}, {keep, (uint64_t)(keep ? samples : 0) * 4, 4, false}};
  const int rc = check_buffers("swin_wattn_block_norm", bufs, 10, 0, 1);
  if (rc != SWIN_WATTN_OK) return rc;
  const cudaError_t e = swin::block_norm_launch(x, f, pre_w, pre_b, post_w, post_b, gate, keep, y, h, tokens, C, samples,
                                                dtype, kind, alpha, eps, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_block_norm");
  ++g_launches;
  return SWIN_WATTN_OK;
}

size_t swin_wattn_block_norm_bwd_workspace_bytes(int tokens, int C) {
  return tokens < 0 || tokens > kMaxLinearTokens || !norm_width(C) ? 0 : swin::block_norm_bwd_workspace_bytes(tokens, C);
}

int swin_wattn_block_norm_bwd(const void* y, const void* f, const void* dh, const void* dy, const float* pre_w,
                              const float* post_w, const float* post_b, const float* gate, const float* keep, void* dx,
                              void* df, float* dpre_w, float* dpre_b, float* dpost_w, float* dpost_b, float* dgate,
                              int tokens, int C, int samples, int dtype, int kind, float alpha, float eps, int accumulate,
                              void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  if (tokens < 0 || !float_dtype(dtype) || (kind != SWIN_WATTN_NORM_LAYER && kind != SWIN_WATTN_NORM_RMS) ||
      !normal_eps(eps) || !std::isfinite(alpha))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (!norm_width(C) || tokens > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (keep != nullptr && (samples < 1 || tokens % samples != 0)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (tokens > 0 && f == nullptr && (post_w != nullptr || gate != nullptr || keep != nullptr))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if ((pre_w == nullptr && (dpre_w != nullptr || dpre_b != nullptr)) ||
      (post_w == nullptr && (post_b != nullptr || dpost_w != nullptr || dpost_b != nullptr)) ||
      (gate == nullptr && dgate != nullptr))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (tokens > 0) {
    if ((dh == nullptr) != (pre_w == nullptr) || (df == nullptr) != (f == nullptr) || dx == nullptr ||
        (pre_w != nullptr && y == nullptr) || (dh == nullptr && dy == nullptr) || workspace == nullptr)
      return SWIN_WATTN_ERR_INVALID_ARG;
    if (workspace_bytes < swin::block_norm_bwd_workspace_bytes(tokens, C)) {
      swin::set_last_error("swin_wattn_block_norm_bwd: workspace smaller than "
                           "swin_wattn_block_norm_bwd_workspace_bytes(tokens, C)");
      return SWIN_WATTN_ERR_INVALID_ARG;
    }
  }
  float* const sums[] = {dpre_w, dpre_b, dpost_w, dpost_b, dgate};
  const bool wanted = std::any_of(sums, sums + 5, [](float* g) { return g != nullptr; });
  if (tokens == 0 && !wanted) return SWIN_WATTN_OK;
  auto live = [&](const void* ptr) { return tokens > 0 ? ptr : nullptr; };
  const uint64_t n = (uint64_t)tokens * C, stream_bytes = n * (dtype == SWIN_WATTN_FP32 ? 4 : 2), c4 = (uint64_t)C * 4;
  const Buffer bufs[] = {{live(dy), stream_bytes, 16, false}, {live(dx), stream_bytes, 16, true},
                         {live(y), stream_bytes, 16, false}, {live(f), n * 2, 16, false}, {live(dh), n * 2, 16, false},
                         {live(df), n * 2, 16, true}, {pre_w, c4, 4, false}, {post_w, c4, 4, false}, {post_b, c4, 4, false},
                         {gate, c4, 4, false}, {live(keep), (uint64_t)(keep ? samples : 0) * 4, 4, false},
                         {dpre_w, c4, 4, true}, {dpre_b, c4, 4, true}, {dpost_w, c4, 4, true}, {dpost_b, c4, 4, true},
                         {dgate, c4, 4, true}, {live(workspace), workspace_bytes, 256, true}};
  const int rc = check_buffers("swin_wattn_block_norm_bwd", bufs, 17, 0, 1);
  if (rc != SWIN_WATTN_OK) return rc;
  const cudaError_t e = swin::block_norm_bwd_launch(y, f, dh, dy, pre_w, post_w, post_b, gate, keep, dx, df, dpre_w, dpre_b,
                                                    dpost_w, dpost_b, dgate, tokens, C, samples, dtype, kind, alpha, eps,
                                                    accumulate, workspace, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_block_norm_bwd");
  g_launches += (tokens > 0) + wanted;
  return SWIN_WATTN_OK;
}

static bool clip_sizes(const int64_t* sizes, const int* dtypes, int count) {
  if (count < 0 || count > 1 << 20 || (count > 0 && (sizes == nullptr || dtypes == nullptr))) return false;
  for (int i = 0; i < count; ++i)
    if (sizes[i] < 0 || sizes[i] > (int64_t)1 << 40 || !float_dtype(dtypes[i])) return false;
  return true;
}

size_t swin_wattn_clip_list_bytes(const int64_t* sizes, const int* dtypes, int count) {
  return clip_sizes(sizes, dtypes, count) ? std::max<size_t>(256, swin::clip_piece_count(sizes, count) * sizeof(swin::ClipPiece)) : 0;
}

int swin_wattn_clip_plan(swin_wattn_clip_t* plan, const void* const* grads, void* const* outs, const int64_t* sizes,
                         const int* dtypes, int count, void* list, size_t list_bytes, struct CUstream_st* stream) {
  if (plan == nullptr) return SWIN_WATTN_ERR_INVALID_ARG;
  *plan = nullptr;
  if (!clip_sizes(sizes, dtypes, count) || list == nullptr || (count > 0 && (grads == nullptr || outs == nullptr)))
    return SWIN_WATTN_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (sizes[i] > 0 && (grads[i] == nullptr || outs[i] == nullptr)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (list_bytes < swin_wattn_clip_list_bytes(sizes, dtypes, count)) {
    swin::set_last_error("swin_wattn_clip_plan: list smaller than swin_wattn_clip_list_bytes(sizes, dtypes, count)");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  try {
    struct Span {
      uint64_t begin, end;
      bool written;
    };
    std::vector<Span> spans;
    int rc = check_on_device(list, 256, dev);
    if (rc != SWIN_WATTN_OK) return rc;
    spans.push_back({reinterpret_cast<uintptr_t>(list), reinterpret_cast<uintptr_t>(list) + list_bytes, true});
    for (int i = 0; i < count; ++i) {
      if (sizes[i] == 0) continue;
      const uint64_t elem = dtypes[i] == SWIN_WATTN_FP32 ? 4 : 2, bytes = (uint64_t)sizes[i] * elem;
      for (const void* ptr : {grads[i], (const void*)outs[i]}) {
        if ((rc = check_on_device(ptr, elem, dev)) != SWIN_WATTN_OK) return rc;
      }
      const uint64_t in = reinterpret_cast<uintptr_t>(grads[i]), out = reinterpret_cast<uintptr_t>(outs[i]);
      spans.push_back({out, out + bytes, true});
      if (in != out) spans.push_back({in, in + bytes, false});
    }
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
    uint64_t end_any = 0, end_written = 0;
    for (const Span& s : spans) {
      if (s.begin < (s.written ? end_any : end_written)) {
        swin::set_last_error("swin_wattn_clip_plan: overlapping tensors");
        return SWIN_WATTN_ERR_INVALID_ARG;
      }
      end_any = std::max(end_any, s.end);
      if (s.written) end_written = std::max(end_written, s.end);
    }
    std::vector<swin::ClipPiece> pieces;
    std::unique_ptr<swin_wattn_clip_s> pl(new swin_wattn_clip_s{{}, static_cast<const swin::ClipPiece*>(list), {}, dev});
    for (const Span& s : spans) {
      if (pl->spans.empty() || s.begin > pl->spans.back().second)
        pl->spans.push_back({s.begin, s.end});
      else
        pl->spans.back().second = std::max(pl->spans.back().second, s.end);
    }
    swin::clip_pieces(grads, outs, sizes, dtypes, count, &pieces, &pl->shape);
    if (!pieces.empty()) {
      const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
      cudaError_t e = cudaMemcpyAsync(list, pieces.data(), pieces.size() * sizeof(swin::ClipPiece), cudaMemcpyHostToDevice, st);
      if (e == cudaSuccess) e = cudaStreamSynchronize(st);
      if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_clip_plan");
    }
    std::lock_guard<std::mutex> lk(g_plans_mu);
    g_clips.insert(pl.get());
    *plan = pl.release();
  } catch (...) {
    swin::set_last_error("swin_wattn_clip_plan: out of host memory");
    return SWIN_WATTN_ERR_CUDA;
  }
  return SWIN_WATTN_OK;
}

size_t swin_wattn_clip_workspace_bytes(void) {
  return swin::clip_workspace_bytes();
}

int swin_wattn_clip_grad_norm(swin_wattn_clip_t plan, float max_norm, float scale, float eps, float* norm, void* workspace,
                              size_t workspace_bytes, struct CUstream_st* stream) {
  int rc = check_clip(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  if (!(max_norm >= 0.0f) || !std::isfinite(max_norm) || !(scale >= FLT_MIN) || !std::isfinite(scale) || !(eps >= 0.0f) ||
      !std::isfinite(eps) || workspace == nullptr)
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (workspace_bytes < swin::clip_workspace_bytes()) {
    swin::set_last_error("swin_wattn_clip_grad_norm: workspace smaller than swin_wattn_clip_workspace_bytes()");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != plan->device) {
    cudaGetLastError();
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  const Buffer bufs[] = {{norm, 4, 4, true}, {workspace, workspace_bytes, 256, true}};
  if ((rc = check_buffers("swin_wattn_clip_grad_norm", bufs, 2)) != SWIN_WATTN_OK) return rc;
  for (const Buffer& b : bufs) {  // against the plan's tensors: the last one that begins before the buffer ends
    if (b.ptr == nullptr) continue;
    const uint64_t p = reinterpret_cast<uintptr_t>(b.ptr);
    auto it = std::lower_bound(plan->spans.begin(), plan->spans.end(), std::make_pair(p + b.bytes, (uint64_t)0));
    if (it != plan->spans.begin() && std::prev(it)->second > p) {
      swin::set_last_error("swin_wattn_clip_grad_norm: norm or workspace overlaps a tensor of the plan");
      return SWIN_WATTN_ERR_INVALID_ARG;
    }
  }
  const cudaError_t e = swin::clip_launch(plan->list, plan->shape, max_norm, scale, eps, norm, workspace,
                                          reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_clip_grad_norm");
  g_launches += swin::clip_launches(plan->shape);
  return SWIN_WATTN_OK;
}

int swin_wattn_clip_destroy(swin_wattn_clip_t plan) {
  if (plan == nullptr) return SWIN_WATTN_OK;
  {
    std::lock_guard<std::mutex> lk(g_plans_mu);
    if (g_clips.erase(plan) == 0) return SWIN_WATTN_ERR_BAD_PLAN;
  }
  delete plan;
  return SWIN_WATTN_OK;
}

size_t swin_wattn_fp4_scale_bytes(int rows, int K, int format) {
  return rows < 0 || rows > kMaxLinearTokens || !fp4_width(K) || !fp4_format(format) ? 0 : swin::fp4::scale_bytes(rows, K, format);
}
size_t swin_wattn_fp4_workspace_bytes(void) { return swin::fp4_workspace_bytes(); }

int swin_wattn_fp4_quantize(const void* x, void* codes, void* scales, float* tensor_scale, int rows, int K, int format,
                            int dtype, int scale_given, void* workspace, size_t workspace_bytes,
                            struct CUstream_st* stream) {
  if (rows < 0 || !fp4_format(format) || !float_dtype(dtype)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (!fp4_width(K) || rows > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  const bool nv = format == SWIN_WATTN_NVFP4, own = nv && !scale_given;
  if (nv != (tensor_scale != nullptr) || (own && (workspace == nullptr || workspace_bytes < swin::fp4_workspace_bytes())))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (rows > 0 && (x == nullptr || codes == nullptr || scales == nullptr)) return SWIN_WATTN_ERR_INVALID_ARG;
  if (rows == 0 && !own) return SWIN_WATTN_OK;
  auto live = [&](const void* ptr) { return rows > 0 ? ptr : nullptr; };
  const uint64_t n = (uint64_t)rows * K;
  const Buffer bufs[] = {{live(x), n * (dtype == SWIN_WATTN_FP32 ? 4 : 2), 16, false}, {live(codes), n / 2, 16, true},
                         {live(scales), swin::fp4::scale_bytes(rows, K, format), 16, true}, {tensor_scale, 4, 4, own},
                         {own ? workspace : nullptr, workspace_bytes, 256, true}};
  const int rc = check_buffers("swin_wattn_fp4_quantize", bufs, 5);
  if (rc != SWIN_WATTN_OK) return rc;
  const cudaError_t e = swin::fp4_quantize_launch(x, codes, scales, tensor_scale, rows, K, format, dtype, scale_given != 0,
                                                  workspace, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_fp4_quantize");
  g_launches += rows == 0 ? 1 : own ? 2 : 1;
  return SWIN_WATTN_OK;
}

int swin_wattn_fp4_dequantize(const void* codes, const void* scales, const float* tensor_scale, void* out, int rows, int K,
                              int format, int dtype, struct CUstream_st* stream) {
  if (rows < 0 || !fp4_format(format) || !float_dtype(dtype) || (format == SWIN_WATTN_NVFP4) != (tensor_scale != nullptr))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (!fp4_width(K) || rows > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (rows == 0) return SWIN_WATTN_OK;
  if (codes == nullptr || scales == nullptr || out == nullptr) return SWIN_WATTN_ERR_INVALID_ARG;
  const uint64_t n = (uint64_t)rows * K;
  const Buffer bufs[] = {{codes, n / 2, 16, false}, {scales, swin::fp4::scale_bytes(rows, K, format), 16, false},
                         {tensor_scale, 4, 4, false}, {out, n * (dtype == SWIN_WATTN_FP32 ? 4 : 2), 16, true}};
  const int rc = check_buffers("swin_wattn_fp4_dequantize", bufs, 4);
  if (rc != SWIN_WATTN_OK) return rc;
  const cudaError_t e = swin::fp4_dequantize_launch(codes, scales, tensor_scale, out, rows, K, format, dtype,
                                                    reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_fp4_dequantize");
  ++g_launches;
  return SWIN_WATTN_OK;
}

int swin_wattn_linear_fp4(const void* x_codes, const void* x_scales, const float* x_tensor_scale, const void* w_codes,
                          const void* w_scales, const float* w_tensor_scale, const float* b, const void* residual, void* y,
                          int tokens, int K, int N, int format, int act, int* status, struct CUstream_st* stream) {
  const bool nv = format == SWIN_WATTN_NVFP4;
  if (tokens < 0 || !known_act(act) || !fp4_format(format) || nv != (x_tensor_scale != nullptr) ||
      nv != (w_tensor_scale != nullptr))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (!fp4_width(K) || !linear_width(N) || tokens > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return SWIN_WATTN_OK;
  if (x_codes == nullptr || x_scales == nullptr || w_codes == nullptr || w_scales == nullptr || y == nullptr)
    return SWIN_WATTN_ERR_INVALID_ARG;
  const uint64_t T = (uint64_t)tokens;
  const Buffer bufs[] = {{residual, T * N * 2, 16, false}, {y, T * N * 2, 16, true}, {x_codes, T * K / 2, 16, false},
                         {x_scales, swin::fp4::scale_bytes(tokens, K, format), 16, false}, {x_tensor_scale, 4, 4, false},
                         {w_codes, (uint64_t)N * K / 2, 16, false}, {w_scales, swin::fp4::scale_bytes(N, K, format), 16, false},
                         {w_tensor_scale, 4, 4, false}, {b, (uint64_t)N * 4, 4, false}, {status, 4, 4, true}};
  const int rc = check_buffers("swin_wattn_linear_fp4", bufs, 10, 0, 1);
  if (rc != SWIN_WATTN_OK) return rc;
  const cudaError_t e = swin::linear_fp4_launch({x_codes, x_scales, x_tensor_scale}, {w_codes, w_scales, w_tensor_scale}, b,
                                                residual, y, tokens, K, N, format, act, status,
                                                reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_linear_fp4");
  ++g_launches;
  return SWIN_WATTN_OK;
}

// The workspace of swin_wattn_linear_fp4_of: codes, scales, the tensor's scale, and what finding it takes.
struct Fp4Workspace {
  size_t scales, tensor_scale, scratch, bytes;
};
static Fp4Workspace fp4_workspace(int tokens, int K, int format) {
  Fp4Workspace w;
  w.scales = ((uint64_t)tokens * K / 2 + 255) / 256 * 256;
  w.tensor_scale = w.scales + swin::fp4::scale_bytes(tokens, K, format);
  w.scratch = w.tensor_scale + 256;
  w.bytes = w.scratch + swin::fp4_workspace_bytes();
  return w;
}

// Whether the product quantises x itself: there is no scale to take from all of x first.
static bool fp4_in_product(int tokens, int K, int N, int format, bool scale_given) {
  return (format != SWIN_WATTN_NVFP4 || scale_given) && swin::linear_fp4_quantizes(tokens, K, N, format);
}

size_t swin_wattn_linear_fp4_workspace_bytes(int tokens, int K, int N, int format, int scale_given) {
  if (tokens <= 0 || tokens > kMaxLinearTokens || !fp4_width(K) || !linear_width(N) || !fp4_format(format)) return 0;
  return fp4_in_product(tokens, K, N, format, scale_given != 0) ? 0 : fp4_workspace(tokens, K, format).bytes;
}

int swin_wattn_linear_fp4_of(const void* x, const float* x_tensor_scale, const void* w_codes, const void* w_scales,
                             const float* w_tensor_scale, const float* b, const void* residual, void* y, int tokens, int K,
                             int N, int format, int dtype, int act, void* workspace, size_t workspace_bytes, int* status,
                             struct CUstream_st* stream) {
  const bool nv = format == SWIN_WATTN_NVFP4, given = x_tensor_scale != nullptr;
  if (tokens < 0 || !known_act(act) || !fp4_format(format) || !float_dtype(dtype) || (given && !nv) ||
      nv != (w_tensor_scale != nullptr))
    return SWIN_WATTN_ERR_INVALID_ARG;
  if (!fp4_width(K) || !linear_width(N) || tokens > kMaxLinearTokens) return SWIN_WATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return SWIN_WATTN_OK;
  const bool in_product = fp4_in_product(tokens, K, N, format, given);
  if (in_product) workspace = nullptr;  // (not looked at)
  if (x == nullptr || w_codes == nullptr || w_scales == nullptr || y == nullptr || (!in_product && workspace == nullptr))
    return SWIN_WATTN_ERR_INVALID_ARG;
  const Fp4Workspace ws = fp4_workspace(tokens, K, format);
  if (!in_product && workspace_bytes < ws.bytes) {
    swin::set_last_error("swin_wattn_linear_fp4_of: workspace smaller than "
                         "swin_wattn_linear_fp4_workspace_bytes(tokens, K, N, format, scale_given)");
    return SWIN_WATTN_ERR_INVALID_ARG;
  }
  const uint64_t T = (uint64_t)tokens;
  const Buffer bufs[] = {{residual, T * N * 2, 16, false}, {y, T * N * 2, 16, true},
                         {x, T * K * (dtype == SWIN_WATTN_FP32 ? 4 : 2), 16, false}, {x_tensor_scale, 4, 4, false},
                         {w_codes, (uint64_t)N * K / 2, 16, false}, {w_scales, swin::fp4::scale_bytes(N, K, format), 16, false},
                         {w_tensor_scale, 4, 4, false}, {b, (uint64_t)N * 4, 4, false}, {status, 4, 4, true},
                         {workspace, workspace_bytes, 256, true}};
  const int rc = check_buffers("swin_wattn_linear_fp4_of", bufs, 10, 0, 1);
  if (rc != SWIN_WATTN_OK) return rc;
  unsigned char* at = static_cast<unsigned char*>(workspace);
  float* scale = !nv ? nullptr : given ? const_cast<float*>(x_tensor_scale) : reinterpret_cast<float*>(at + ws.tensor_scale);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (in_product) {
    const cudaError_t e = swin::linear_fp4_of_few(x, dtype, x_tensor_scale, {w_codes, w_scales, w_tensor_scale}, b, residual, y,
                                                  tokens, K, N, format, act, status, st);
    if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_linear_fp4_of");
    ++g_launches;
    return SWIN_WATTN_OK;
  }
  cudaError_t e = swin::fp4_quantize_launch(x, at, at + ws.scales, scale, tokens, K, format, dtype, given, at + ws.scratch, st);
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_linear_fp4_of");
  g_launches += nv && !given ? 2 : 1;
  e = swin::linear_fp4_launch({at, at + ws.scales, scale}, {w_codes, w_scales, w_tensor_scale}, b, residual, y, tokens, K, N,
                              format, act, status, st);
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_linear_fp4_of");
  ++g_launches;
  return SWIN_WATTN_OK;
}

int swin_wattn_set_fwd_kernel(swin_wattn_plan_t plan, int kernel) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  if (kernel != SWIN_WATTN_KERNEL_AUTO && kernel != SWIN_WATTN_KERNEL_MMA_SYNC &&
      kernel != SWIN_WATTN_KERNEL_TCGEN05)
    return SWIN_WATTN_ERR_INVALID_ARG;
  swin::Plan& p = plan->p;
  const int old = p.fwd_kernel;
  p.fwd_kernel = kernel;
  swin::FwdLaunch L;
  cudaError_t e = swin::fwd_config(p, &L);
  if (e == cudaErrorNotSupported) {
    p.fwd_kernel = old;
    return SWIN_WATTN_ERR_UNSUPPORTED;
  }
  if (e != cudaSuccess) {
    p.fwd_kernel = old;
    return cuda_fail(e, "swin_wattn_set_fwd_kernel");
  }
  plan->fwd = L;
  return SWIN_WATTN_OK;
}

int swin_wattn_fwd_kernel(swin_wattn_plan_t plan) {
  if (check_plan(plan) != SWIN_WATTN_OK) return -1;
  return plan->fwd.tc ? SWIN_WATTN_KERNEL_TCGEN05 : SWIN_WATTN_KERNEL_MMA_SYNC;
}

int swin_wattn_set_bwd_kernel(swin_wattn_plan_t plan, int kernel) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  if (kernel != SWIN_WATTN_KERNEL_AUTO && kernel != SWIN_WATTN_KERNEL_MMA_SYNC &&
      kernel != SWIN_WATTN_KERNEL_TCGEN05)
    return SWIN_WATTN_ERR_INVALID_ARG;
  swin::Plan& p = plan->p;
  const int old = p.bwd_kernel;
  p.bwd_kernel = kernel;
  swin::BwdLaunch L;
  cudaError_t e = swin::bwd_config(p, &L);
  if (e == cudaErrorNotSupported || (e == cudaSuccess && L.grid == 0 && p.B > 0)) {
    p.bwd_kernel = old;
    return SWIN_WATTN_ERR_UNSUPPORTED;
  }
  if (e != cudaSuccess) {
    p.bwd_kernel = old;
    return cuda_fail(e, "swin_wattn_set_bwd_kernel");
  }
  plan->bwd = L;
  return SWIN_WATTN_OK;
}

int swin_wattn_bwd_kernel(swin_wattn_plan_t plan) {
  if (check_plan(plan) != SWIN_WATTN_OK) return -1;
  return plan->bwd.tc ? SWIN_WATTN_KERNEL_TCGEN05 : SWIN_WATTN_KERNEL_MMA_SYNC;
}

int swin_wattn_device_status(swin_wattn_plan_t plan, struct CUstream_st* stream) {
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, plan->p.err, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && word != 0) e = cudaMemsetAsync(plan->p.err, 0, sizeof(int), st);
  if (e == cudaSuccess && word != 0) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "swin_wattn_device_status");
  if (word != 0) {
    swin::set_last_error("a bounded device wait ran out (tensor-core completion never arrived)");
    return SWIN_WATTN_ERR_TIMEOUT;
  }
  return SWIN_WATTN_OK;
}

int swin_wattn_destroy(swin_wattn_plan_t plan) {
  if (plan == nullptr) return SWIN_WATTN_OK;
  int rc = check_plan(plan);
  if (rc != SWIN_WATTN_OK) return rc;
  {
    std::lock_guard<std::mutex> lk(g_plans_mu);
    g_plans.erase(plan);
  }
  cudaError_t e = cudaDeviceSynchronize();
  plan->p.magic = 0;
  free_pipe(plan->pipe);
  free_plan_buffers(plan->p);
  delete plan;
  return e == cudaSuccess ? SWIN_WATTN_OK : cuda_fail(e, "swin_wattn_destroy");
}

}  // extern "C"
