// host_common.h -- what the host-side translation units share: the calling
// thread's error message, the driver's tensor-map encoder, the environment
// hooks, the plan object and the registry of live plans.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>
#include <unordered_set>

#include "../../include/gemm_epi.h"
#include "few_rows.cuh"
#include "kernel_table.h"

namespace ge_host {

inline thread_local std::string g_last_error;

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

// The error stays with this call: the runtime would hand it to the next launch that asks for the last one.
inline int cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(GEMM_EPI_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

// ----------------------------------------------------- driver entry points
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Fault-injection hooks for the tests take effect only while
// GEMM_EPI_TEST_HOOKS=1 is set as well, so that one stray variable inherited
// by a production process cannot make its plans stall or fail.
inline bool test_hooks_on() {
  const char* f = getenv("GEMM_EPI_TEST_HOOKS");
  return f && atoi(f) == 1;
}
inline bool test_hook(const char* name) {
  const char* f = test_hooks_on() ? getenv(name) : nullptr;
  return f && atoi(f) != 0;
}

// GEMM_EPI_INJECT_ENCODE_FAILURE makes every tensor-map encode fail, so an
// execute call must return GEMM_EPI_ERR_CUDA before it launches anything.
inline bool inject_encode_failure() { return test_hook("GEMM_EPI_INJECT_ENCODE_FAILURE"); }

// The watchdog settings a launch carries: the limit of each bounded wait
// (2 s; GEMM_EPI_WAIT_TIMEOUT_MS overrides) and, for the watchdog tests,
// GEMM_EPI_INJECT_STALL -- the MMA issuer withholds its first tile's
// completion signal, so the epilogue's wait runs out and the kernel reports
// ERR_TIMEOUT (2, grouped and microscaled plans, 4-bit weights and gated few-row plans: one CTA
// of the first launch only). Read when a plan is created and on every call of the allocation-free
// entry point.
struct WatchdogEnv {
  uint64_t timeout_ns = 2000000000ull;
  int inject_stall = 0;
};
inline WatchdogEnv watchdog_env() {
  WatchdogEnv w;
  if (const char* t = getenv("GEMM_EPI_WAIT_TIMEOUT_MS")) {
    const long long ms = atoll(t);
    if (ms > 0) w.timeout_ns = (uint64_t)ms * 1000000ull;
  }
  if (test_hook("GEMM_EPI_INJECT_STALL")) w.inject_stall = atoi(getenv("GEMM_EPI_INJECT_STALL")) == 2 ? 2 : 1;
  return w;
}

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}


struct TileCfg {
  int BN = 256, stages = 4;
  ge_inst::TileKernelFn fn = nullptr;
  uint32_t smem = 0;
  bool pair = false;  // CTA-pair kernel, launched in clusters of 2
  int threads = 192;
};

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

struct SkinnyCfg {
  int TP = 16;
  int KPS = 1;  // 64-deep k-blocks per pipeline stage
  ge_inst::SkinnyKernelFn fn = nullptr;
  uint32_t smem = 0;
  int stages = 0;
};

// A plan of products grouped by expert, or of a microscaled product.
struct GroupedCfg {
  ge_inst::GroupedKernelFn fn = nullptr;
  ge_inst::MxKernelFn mx_fn = nullptr;  // kind == 2
  uint32_t smem = 0;
  int threads = 0, stages = 0;
  int TR = 0, BK = 64;  // rows of a tile; k per stage
  bool pair = false;
  int E = 0 /* 0: no groups (kind 2) */, n_ft = 0, n_kt = 0, group = 1;
  int slices = 1;  // WGRAD: row slices of the optional bias gradient
};

// A gated layer's kernel whose warps work alone, if there is a function.
struct GatedFewCfg {
  ge_inst::GatedFewKernelFn fn = nullptr;
  uint32_t smem = 0;
  int grid = 0;
  ge::FewSplit few = {};
};

// A plan of few rows times 4-bit weights.
struct W4Cfg {
  ge_inst::W4KernelFn fn = nullptr;
  ge_inst::W4FewInstance few = {};       // the kernel of warps alone, if it has threads
  ge::FewSplit few_split = {};
  uint32_t smem = 0;
  int threads = 0, tp = 0, row_blocks = 1, tiles = 0, kt = 0, grid = 0, max_segs = 1, stages = 0;
};

// Row-major matrices of bytes, 16-bit or 32-bit elements: `d2` of them, `d1`
// rows of `d0` contiguous elements each; boxes of b0 x b1.
inline int encode_3d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                     uint32_t b0, uint32_t b1, const char* name,
                     CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(GEMM_EPI_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (inject_encode_failure()) return fail(GEMM_EPI_ERR_CUDA, "injected tensor map encode failure");
  const uint64_t size = type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 1 : type == CU_TENSOR_MAP_DATA_TYPE_UINT16 ? 2 : 4;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {d0 * size, d0 * size * d1};
  const cuuint32_t box[3] = {b0, b1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(GEMM_EPI_ERR_CUDA, "tensor map encode for %s failed (CUresult %d)", name, (int)r);
  return GEMM_EPI_OK;
}

// Counters of a new workspace set to zero, and done with when this returns:
// the plan's first call may run on any stream, and a memset on the legacy
// stream, which could be behind, is not waited for by all of them. On a stream
// of the library's own, one a device (making one a plan took 200 us).
inline cudaError_t zero_counts(int* counts, size_t n) {
  constexpr int kMax = 64;
  static std::atomic<cudaStream_t> kept[kMax];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool keep = dev >= 0 && dev < kMax;
  cudaStream_t s = keep ? kept[dev].load() : nullptr;
  if (!s) {
    e = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
    if (e != cudaSuccess) return e;
  }
  e = cudaMemsetAsync(counts, 0, sizeof(int) * n, s);
  const cudaError_t done = cudaStreamSynchronize(s);
  cudaStream_t none = nullptr;
  if (!keep || (kept[dev].load() != s && !kept[dev].compare_exchange_strong(none, s))) cudaStreamDestroy(s);
  return e != cudaSuccess ? e : done;
}

// The current device's number and SM count; an error unless it is a B200. The
// device's properties are asked for once (they never change).
inline int require_b200(int* dev, int* sms) {
  constexpr int kMax = 64;
  static std::atomic<int> known[kMax];  // 0: not asked yet; else 1 + SM count, negative if no B200
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  int v = *dev >= 0 && *dev < kMax ? known[*dev].load(std::memory_order_relaxed) : 0;
  if (v == 0) {
    int major = 0, minor = 0, n = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev);
    v = major == 10 && minor == 0 && n > 0 ? 1 + n : -(major * 16 + minor) - 1;
    if (*dev >= 0 && *dev < kMax) known[*dev].store(v, std::memory_order_relaxed);
  }
  if (v < 0)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "device %d has compute capability %d.%d; this library needs 10.0 (sm_100a)", *dev,
                (-v - 1) / 16, (-v - 1) % 16);
  *sms = v - 1;
  return GEMM_EPI_OK;
}

// A launch configuration: clusters of two for CTA pairs, and programmatic
// serialization, so that a kernel's set-up (barriers, tensor memory) overlaps
// the end of the kernel before it; the kernels wait for it before they touch
// global memory (ge::wait_for_inputs).
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Launch(dim3 grid, int threads, size_t smem, bool pair, cudaStream_t s) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pair ? 2 : 1;
  }
  Launch(int grid, int threads, size_t smem, bool pair, cudaStream_t s)
      : Launch(dim3((unsigned)grid, 1, 1), threads, smem, pair, s) {}
  Launch(const Launch&) = delete;
  Launch& operator=(const Launch&) = delete;
};

// Clusters of `size` CTAs of this kernel that the device holds at once; one per `size`
// SMs if the query fails.
inline int resident_clusters(const void* fn, int size, int threads, uint32_t smem, int sms) {
  Launch l(sms / size * size, threads, smem, true, nullptr);
  l.attr[1].val.clusterDim.x = (unsigned)size;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &l.cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return sms / size;
  }
  return n < sms / size ? n : sms / size;
}
inline int resident_pairs(const void* fn, int threads, uint32_t smem, int sms) {
  return resident_clusters(fn, 2, threads, smem, sms);
}

// Makes `device` current for the calls of one entry point and puts the
// caller's device back, so that a plan runs on its own device from any.
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    if (cudaGetDevice(&before_) != cudaSuccess) before_ = -1;
    if (before_ != device) changed_ = cudaSetDevice(device) == cudaSuccess;
  }
  ~DeviceScope() {
    if (changed_ && before_ >= 0) cudaSetDevice(before_);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;

 private:
  int before_ = -1;
  bool changed_ = false;
};

}  // namespace ge_host

struct gemm_epi_plan_s {
  int kind = 0;      // 0: one product; 1: products grouped by expert (grouped.cu); 2: microscaled (mx.cu); 3: gated (gated.cu); 4: 4-bit weights (w4.cu)
  int64_t T, N, K;   // the kernels' rows, columns and contraction length
  int64_t uT, uK;    // the caller's T and K (WGRAD: rows = uK, contraction = uT)
  int dtype, epilog;
  int device, num_sms;
  int m_tiles, n_tiles, k_blocks, num_tiles, aux_words, grid, group_m;
  int raster_n = 0;  // tile order by column groups (see choose_raster)
  int pair_split = 0;        // CTA pairs in stream-K mode
  int pair_sk_first = 1;     // stream-K tiles before the whole tiles
  int pair_max_segs = 1;
  float* pair_slots = nullptr;  // stream-K fp32 partials
  int* pair_flags = nullptr;    // stream-K segment counters, zero between launches
  int n_pair_flags = 0;
  size_t pair_bytes = 0;
  ge_host::TileCfg cfg;       // fused kernel
  ge_host::TileCfg cfg_store; // unfused GEMM (plain store)
  float* partials = nullptr;  // DRELU_BGRAD: m_tiles x N
  size_t partial_bytes = 0;
  int* col_tickets = nullptr;  // DRELU_BGRAD on the tile kernels: n_tickets counters
  int n_tickets = 0;
  int* status_host = nullptr;
  int* status_dev = nullptr;
  uint64_t timeout_ns = 0;
  int inject_stall = 0;  // GEMM_EPI_INJECT_STALL at plan time (watchdog tests)
  bool counts_stale = false;  // an interrupted launch may have left counters of this workspace above zero
  int tail_split = 1;    // GEMM_EPI_TAIL_SPLIT=0 keeps whole tiles in the pair kernel's last round
  int bias_f32 = 0;      // gemm_epi_set_bias_f32: the forward bias is fp32
  int w_nk = 0;          // GEMM_EPI_FLAG_W_NK: W / W2 given N x K (K contiguous)
  int out_f32 = 0;       // GEMM_EPI_FLAG_OUT_F32: Y / dZ / dW written as fp32
  int act = 0;           // kind 3, 4: gemm_epi_act
  int no_dbias = 0;      // GEMM_EPI_FLAG_NO_DBIAS
  ge_host::GatedFewCfg gf;  // kind 3
  ge_host::W4Cfg w4;     // kind 4
  int cache_hints = 0;   // few-row kernel: L2 eviction policies on the operand loads (GEMM_EPI_CACHE_HINTS)
  // tensor-map cache
  const void* a_ptr = nullptr;
  const void* b_ptr = nullptr;
  const void* y_ptr = nullptr;
  const void* aux_ptr = nullptr;
  CUtensorMap tmA, tmB, tmY, tmAux;
  // few-row kernel (kernel == 1)
  int kernel = 0;
  ge_host::SkinnyCfg sk;
  int sk_features = 128;  // gated: features of H in a tile
  int sk_grid = 0, sk_kbt = 0, sk_total = 0, sk_max_segs = 1, sk_prefetch = 0;
  float* sk_partials = nullptr;
  int* sk_tickets = nullptr;
  size_t sk_bytes = 0;
  const void* xs_ptr = nullptr;
  CUtensorMap tmXs;  // the row operand with a TP-row box
  const void* ws_ptr = nullptr;
  CUtensorMap tmWs;  // the weight operand with a 64·KPS-row box
  ge_host::GroupedCfg gr;  // kind 1 and 2
  int force_splits = 0;    // GEMM_EPI_FORCE_SPLIT
  int split_items = 0;     // counters in sk_tickets (kind 1, one-CTA tiles: slots of the k split)
  size_t split_bytes = 0;
  int split_k = 1;         // kind 1: the parts of a tile where every expert has the mean number of rows
};

namespace ge_host {

// ---------------------------------------------------------------- registry
inline std::mutex g_mu;
inline std::unordered_set<gemm_epi_plan_s*>& live_plans() {
  static std::unordered_set<gemm_epi_plan_s*> s;
  return s;
}

inline gemm_epi_plan_s* lookup(gemm_epi_plan_t p) {
  std::lock_guard<std::mutex> g(g_mu);
  return live_plans().count(p) ? p : nullptr;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// the live plan of this kind, or NULL with the error set
inline gemm_epi_plan_s* lookup_kind(gemm_epi_plan_t plan, int kind, const char* call, int* code) {
  gemm_epi_plan_s* p = lookup(plan);
  *code = GEMM_EPI_OK;
  if (!p) {
    *code = fail(GEMM_EPI_ERR_INVALID_ARG, "%s: unknown plan", call);
  } else if (p->kind != kind) {
    const char* what[] = {"of one product", "of products grouped by expert", "of a microscaled product", "of a gated layer", "of 4-bit weights"};
    *code = fail(GEMM_EPI_ERR_EPILOG_MISMATCH, "%s called on a plan %s", call, what[p->kind]);
    p = nullptr;
  }
  return p;
}

inline int take_status(gemm_epi_plan_s* p) {
  volatile int* s = p->status_host;
  const int v = *s;
  if (v != 0) {
    *s = 0;
    p->counts_stale = true;
    return fail(GEMM_EPI_ERR_TIMEOUT, "a kernel of this plan gave up waiting (watchdog code 0x%x)", v);
  }
  return GEMM_EPI_OK;
}

// Before a call launches: the report of an earlier run-out, and the counters
// that it left cleared on the call's own stream (the legacy stream orders
// nothing for a stream that does not block on it). While a stream is being
// captured the clearing becomes part of the graph, so it stays due until a call
// that runs.
inline int begin_call(gemm_epi_plan_s* p, cudaStream_t stream) {
  const int rc = take_status(p);
  if (rc || !p->counts_stale) return rc;
  const auto clear = [stream](int* counts, int n) {
    return counts ? cudaMemsetAsync(counts, 0, sizeof(int) * (size_t)n, stream) : cudaSuccess;
  };
  cudaError_t e = clear(p->sk_tickets, p->kind == 0 ? ceil_div(p->N, 128) : p->split_items);
  if (e == cudaSuccess) e = clear(p->col_tickets, p->n_tickets);
  if (e == cudaSuccess) e = clear(p->pair_flags, p->n_pair_flags);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the workspace of an interrupted launch");
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &capture) == cudaSuccess && capture == cudaStreamCaptureStatusNone)
    p->counts_stale = false;
  return GEMM_EPI_OK;
}

}  // namespace ge_host
