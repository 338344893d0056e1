// gated.cu -- C ABI of gated layers: plan validation and kernel choice, TMA
// descriptors, launches.
#include "gated_few.cuh"
#include "host_tiles.h"
#include "skinny_kernel.cuh"

using namespace ge_host;

static_assert(static_cast<int>(GEMM_EPI_GATED) == ge::EPI_GATED && static_cast<int>(GEMM_EPI_DGATED) == ge::EPI_DGATED &&
                  static_cast<int>(GEMM_EPI_SILU) == ge::ACT_SILU && static_cast<int>(GEMM_EPI_GELU) == ge::ACT_GELU &&
                  static_cast<int>(GEMM_EPI_RELU) == ge::ACT_RELU,
              "the public values are the kernels'");

namespace {

ge_inst::GatedInstance instance(bool bf16, bool w_nk, int bn, bool pair, int epi) {
  if (bf16) return w_nk ? ge_inst::gated_bf16_nk(bn, pair, epi) : ge_inst::gated_bf16_mn(bn, pair, epi);
  return w_nk ? ge_inst::gated_f16_nk(bn, pair, epi) : ge_inst::gated_f16_mn(bn, pair, epi);
}

ge_inst::GatedSkinnyInstance skinny_instance(bool bf16, bool w_nk, int tp, int gn) {
  if (bf16) return w_nk ? ge_inst::gated_skinny_bf16_nk(tp, gn) : ge_inst::gated_skinny_bf16_mn(tp, gn);
  return w_nk ? ge_inst::gated_skinny_f16_nk(tp, gn) : ge_inst::gated_skinny_f16_mn(tp, gn);
}

// Accumulator columns that tiles of bn cover: a gated tile is half gate, half up.
int64_t columns(int64_t N, bool forward, int bn) {
  return forward ? (N + bn / 2 - 1) / (bn / 2) * bn : N;
}

// Tiles by the dense plans' estimates (GEMM_EPI_FORCE_BN and _FORCE_KERNEL override
// where there is such an instance): CTA pairs for X of at most 1 GiB where they
// are estimated no slower, also with less than a wave of their tiles (DGATED, fp16,
// us, tiles / pairs: T = 160, K = 4096, N = 11008 40 / 35; T = 1024, K = N = 4096 38.5 /
// 35.5; GATED, T = 300, K = 2048, N = 4096 17.6 / 17.9).
int choose_bn(int64_t T, int64_t N, int64_t K, bool forward, int sms) {
  if (const char* f = getenv("GEMM_EPI_FORCE_BN")) {
    const int v = atoi(f);
    if (v == 128 || v == 256 || (v == 64 && !forward)) return v;
  }
  int best = 256;
  double best_us = est_tile_us(T, columns(N, forward, 256), K, 256, sms);
  for (int bn : {128, 64}) {
    if (forward && bn == 64) break;
    const double us = est_tile_us(T, columns(N, forward, bn), K, bn, sms);
    if (us < best_us * 0.999) {
      best = bn;
      best_us = us;
    }
  }
  return best;
}

bool use_pair(int64_t T, int64_t N, int64_t K, bool forward, int bn, int sms) {
  if (const char* f = getenv("GEMM_EPI_FORCE_KERNEL")) {
    if (!strcmp(f, "tile") || !strcmp(f, "skinny")) return false;
    if (!strcmp(f, "pair")) return T > 32;
  }
  if (T <= 128 || T * K * 2 > ((int64_t)1 << 30)) return false;
  return est_pair_us(T, columns(N, forward, 256), K, sms / 2) <= est_tile_us(T, columns(N, forward, bn), K, bn, sms);
}

// The few-row kernel for T <= 32. Measured (us, few-row / tiles): K = 4096, N =
// 11008, T = 32 31.3 / 35, T = 64 41.8 / 35.2, T = 128 47.9 / 35.5; K = 2048, N = 5632,
// T = 64 25.8 / 13.8.
bool use_skinny(int64_t T) {
  if (const char* f = getenv("GEMM_EPI_FORCE_KERNEL")) {
    if (!strcmp(f, "tile")) return false;
  }
  return T <= 32;
}

// The pre-activations, T x 2N, as rows of two matrices of N columns, in blocks of 32
// rows and 64 bytes: what is stored past column N of one half is cut off.
int encode_halves(CUtensorMap* map, const void* base, int64_t T, int64_t N) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(GEMM_EPI_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (inject_encode_failure()) return fail(GEMM_EPI_ERR_CUDA, "injected tensor map encode failure");
  const cuuint64_t dims[3] = {(cuuint64_t)N, 2, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)N * 2, (cuuint64_t)N * 4};
  const cuuint32_t box[3] = {32, 1, 32};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(GEMM_EPI_ERR_CUDA, "tensor map encode for the pre-activations failed (CUresult %d)", (int)r);
  return GEMM_EPI_OK;
}

void release(gemm_epi_plan_s* p) {
  if (p->partials) cudaFree(p->partials);
  if (p->sk_partials) cudaFree(p->sk_partials);
  if (p->sk_tickets) cudaFree(p->sk_tickets);
  if (p->status_host) cudaFreeHost(p->status_host);
  delete p;
}

// Features of H of a few-row tile (128 where that makes as many tiles as half the SMs), and
// whether the kernel takes whole tiles.
int few_row_features(int64_t N, int sms) { return 2 * ceil_div(N, 128) >= sms ? 128 : 64; }
bool whole_tiles(int64_t N, int sms) {
  const int tiles = ceil_div(N, few_row_features(N, sms));
  return tiles * 2 >= sms && tiles <= sms;
}

// The kernel whose warps work alone, for at most 16 rows of a small weight: it starts 2
// to 3 us sooner, and streams at half the rate of TMA's. By the half tiles of a warp, N x K (K x N), us,
// T = 1, the few-row kernel's behind the stroke:
//   2  K = 1024, N = 2048 4.6 / 6.6        4  K = N = 2048 7.7 / 10.1
//   6  K = 3008, N = 1024 8.5 (9.6) / 10.0, N = 2048 9.4 (10.3) / 11.1
//   7  K = 3584, N = 1024 9.8 (10.7) / 10.0, N = 2048 10.6 (11.5) / 11.5
//   8  one half row a CTA: K = 4096, N = 1024 11.0 (11.8) / 10.0, N = 1536 11.4 (12.2) / 10.9, N = 2360 12.4
//      (13.1) / 11.7; T = 16, N = 1536 12.5 / 11.3
//   8  more half rows a CTA: K = 2048, N = 3000 9.2 (9.4) / 10.5, N = 4096 10.3 (9.5) / 11.6; T = 16 11.5 / 11.9
//  12  K = N = 3000 12.9 / 12.6           20  K = 4096, N = 11008 38.1 / 31.8
// where the few-row kernel has whole tiles 6: K = 1024, N = 5632 8.8 / 7.9, 12: K = 2048 13.9 / 11.3.
// Where a split of the columns over a cluster is estimated fastest (few features, K from 2560
// on), the few-row kernel is faster than with it and than without: K = 4096, N = 512 14.3 split, 10.7 whole
// / 9.0, K = 8192, N = 256 15.8 split / 11.2. So only the override launches clusters here.
bool plan_few(gemm_epi_plan_s* p, bool bf16, cudaError_t* e) {
  if (p->T > 16) return false;
  bool forced = false;
  if (const char* f = getenv("GEMM_EPI_FORCE_KERNEL")) {  // tuning override
    forced = !strcmp(f, "warp");
    if (!strcmp(f, "skinny")) return false;
  }
  const int kt = ceil_div(p->K, 32);
  if ((p->N / 16 + 1) * (int64_t)kt >= (int64_t)1 << 28) return false;  // (32-bit shares)
  // (the grid of the other kernel; a stall needs a wait)
  if (!forced && (getenv("GEMM_EPI_SKINNY_GRID") || p->inject_stall)) return false;
  const ge_inst::GatedFewInstance inst = ge_inst::gated_few(bf16, p->w_nk != 0, (int)p->T);
  *e = cudaFuncSetAttribute(inst.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)inst.smem);
  if (*e != cudaSuccess) return true;
  const FewChoice choice = choose_few((const void*)inst.fn, 32 * ge::kFewWarps, inst.smem, p->N, kt, p->num_sms, 1, 3);
  // (whole tiles are what the other kernel is best at)
  const int64_t most = whole_tiles(p->N, p->num_sms) ? 4 : ceil_div(p->N, 16) <= p->num_sms ? 7 : 8;
  if (!forced && (choice.split > 0 || choice.steps > most)) return false;
  p->gf.fn = inst.fn;
  p->gf.smem = inst.smem;
  p->gf.grid = choice.clusters << choice.split;
  p->gf.few = few_split(choice, p->N, kt);
  p->kernel = 1;
  return true;
}

int run_few(gemm_epi_plan_s* p, const void* X, const void* W, const void* bias, void* H, void* aux, cudaStream_t stream) {
  ge::GatedFewParams k{};
  k.T = (int32_t)p->T;
  k.N = (int32_t)p->N;
  k.K = (int32_t)p->K;
  k.act = p->act;
  k.bias_f32 = p->bias_f32;
  k.out_f32 = p->out_f32;
  k.few = p->gf.few;
  k.X = X;
  k.W = W;
  k.bias = bias;
  k.out = H;
  k.aux_out = aux;
  Launch l(p->gf.grid, 32 * ge::kFewWarps, p->gf.smem, k.few.split > 0, stream);
  l.attr[1].val.clusterDim.x = 1u << k.few.split;
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, p->gf.fn, k);
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "gated few-row launch");
}

// The few-row kernel's schedule: whole tiles where there are between half as many
// as SMs and as many -- of 128 features of H if there are that many, else of 64 -- and
// otherwise equal shares of all k-blocks, at least 256 k each.
cudaError_t plan_skinny(gemm_epi_plan_s* p, bool bf16, int sms) {
  const int tp = p->T <= 16 ? 16 : 32;
  const int gn = few_row_features(p->N, sms);
  const ge_inst::GatedSkinnyInstance inst = skinny_instance(bf16, p->w_nk != 0, tp, gn);
  p->kernel = 1;
  p->sk.TP = tp;
  p->sk.KPS = 2;
  p->sk.fn = inst.fn;
  p->sk.smem = inst.smem;
  p->sk.stages = inst.stages;
  p->sk_features = gn;
  const int n_tiles = ceil_div(p->N, gn);
  p->sk_kbt = ceil_div(p->K, (int64_t)ge::kBK * 2);
  p->sk_total = n_tiles * p->sk_kbt;
  if (whole_tiles(p->N, sms)) {
    p->sk_grid = n_tiles;
  } else {
    const int g = p->sk_total / 2;
    p->sk_grid = g < 1 ? 1 : g < sms ? g : sms;
  }
  if (const char* f = getenv("GEMM_EPI_SKINNY_GRID")) {  // tuning override
    const int v = atoi(f);
    if (v >= 1 && v <= p->sk_total && (int64_t)(p->sk_total + 1) * v < (int64_t(1) << 31)) p->sk_grid = v;
  }
  for (int t = 0; t < n_tiles; ++t) {
    const int64_t first = ge::skinny_owner((int64_t)t * p->sk_kbt, p->sk_grid, p->sk_total);
    const int64_t last = ge::skinny_owner((int64_t)(t + 1) * p->sk_kbt - 1, p->sk_grid, p->sk_total);
    if (last - first + 1 > p->sk_max_segs) p->sk_max_segs = (int)(last - first + 1);
  }
  cudaError_t e = cudaFuncSetAttribute(p->sk.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p->sk.smem);
  if (e != cudaSuccess || p->sk_max_segs == 1) return e;
  p->sk_bytes = (size_t)n_tiles * p->sk_max_segs * (gn / 64) * tp * 128 * sizeof(float);
  e = cudaMalloc((void**)&p->sk_partials, p->sk_bytes);
  if (e != cudaSuccess) return e;
  e = cudaMalloc((void**)&p->sk_tickets, sizeof(int) * (size_t)n_tiles);
  if (e != cudaSuccess) return e;
  p->split_items = n_tiles;
  p->sk_bytes += sizeof(int) * (size_t)n_tiles;
  return zero_counts(p->sk_tickets, (size_t)n_tiles);
}

cudaError_t plan_tiles(gemm_epi_plan_s* p, bool bf16, bool forward, int sms) {
  int bn = choose_bn(p->T, p->N, p->K, forward, sms);
  const bool pair = use_pair(p->T, p->N, p->K, forward, bn, sms);
  if (pair) bn = 256;
  const int bno = forward ? bn / 2 : bn;
  const ge_inst::GatedInstance inst = instance(bf16, p->w_nk != 0, bn, pair, forward ? ge::EPI_GATED : ge::EPI_DGATED);
  p->kernel = pair ? 2 : 0;
  p->cfg.BN = bn;
  p->cfg.stages = inst.stages;
  p->cfg.fn = inst.fn;
  p->cfg.smem = inst.smem;
  p->cfg.pair = pair;
  p->cfg.threads = inst.threads;
  p->m_tiles = ceil_div(p->T, ge::kBM);
  p->n_tiles = ceil_div(p->N, bno);
  p->k_blocks = ceil_div(p->K, ge::kBK);
  p->num_tiles = p->m_tiles * p->n_tiles;
  const Raster raster = choose_raster(p->T, columns(p->N, forward, bn), p->K, pair ? 2 * ge::kBM : ge::kBM, bn);
  p->group_m = raster.group;
  p->raster_n = raster.by_n;
  if (const char* f = getenv("GEMM_EPI_TAIL_SPLIT")) p->tail_split = atoi(f) != 0;
  cudaError_t e = cudaFuncSetAttribute(p->cfg.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p->cfg.smem);
  if (e != cudaSuccess) return e;
  if (pair) {
    const int tiles = ceil_div(p->T, 256) * p->n_tiles;
    const int pairs = resident_pairs((const void*)p->cfg.fn, p->cfg.threads, p->cfg.smem, sms);
    // (at most half as many tiles as pairs: a pair for each half of a tile)
    p->grid = 2 * (p->tail_split && 2 * tiles <= pairs ? 2 * tiles : tiles < pairs ? tiles : pairs);
  } else {
    p->grid = p->num_tiles < sms ? p->num_tiles : sms;
  }
  if (forward || p->no_dbias) return cudaSuccess;
  // the bias gradient's partial sums, a row for each 32 of T
  p->partial_bytes = (size_t)ceil_div(p->T, 32) * 2 * (size_t)p->N * sizeof(float);
  if (test_hook("GEMM_EPI_INJECT_PLAN_ALLOC_FAILURE")) return cudaErrorMemoryAllocation;
  return cudaMalloc((void**)&p->partials, p->partial_bytes);
}

gemm_epi_plan_t make_plan(int64_t T, int64_t N, int64_t K, gemm_epi_dtype dtype, gemm_epi_gated_epilog epilog,
                          gemm_epi_act act, uint32_t flags) {
  const uint32_t known = GEMM_EPI_FLAG_W_NK | GEMM_EPI_FLAG_OUT_F32 | (epilog == GEMM_EPI_DGATED ? GEMM_EPI_FLAG_NO_DBIAS : 0u);
  if ((flags & ~known) != 0) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown plan flags 0x%x", flags & ~known);
    return nullptr;
  }
  if (T < 1 || N < 8 || K < 8 || (N % 8) != 0 || (K % 8) != 0) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "bad shape T=%lld N=%lld K=%lld (need T>=1, N,K>=8 and multiples of 8)", (long long)T,
         (long long)N, (long long)K);
    return nullptr;
  }
  if (T > (int64_t)1 << 30 || N > (int64_t)1 << 23 || K > (int64_t)1 << 24 || T * N > ((int64_t)1 << 39) ||
      ((T + 127) / 128) * ((N + 63) / 64) >= ((int64_t)1 << 31) - 65536) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "shape too large for 32-bit tile coordinates");
    return nullptr;
  }
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    return nullptr;
  }
  if (epilog != GEMM_EPI_GATED && epilog != GEMM_EPI_GATED_AUX && epilog != GEMM_EPI_DGATED) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "epilog %d is none of a gated layer (GATED, GATED_AUX, DGATED)", (int)epilog);
    return nullptr;
  }
  if (act != GEMM_EPI_SILU && act != GEMM_EPI_GELU && act != GEMM_EPI_RELU) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    return nullptr;
  }
  int dev = 0, sms = 0;
  if (require_b200(&dev, &sms)) return nullptr;
  auto* p = new gemm_epi_plan_s();
  p->kind = 3;
  p->uT = p->T = T;
  p->uK = p->K = K;
  p->N = N;
  p->dtype = dtype;
  p->epilog = epilog;
  p->act = act;
  p->w_nk = (flags & GEMM_EPI_FLAG_W_NK) ? 1 : 0;
  p->out_f32 = (flags & GEMM_EPI_FLAG_OUT_F32) ? 1 : 0;
  p->no_dbias = (flags & GEMM_EPI_FLAG_NO_DBIAS) ? 1 : 0;
  p->device = dev;
  p->num_sms = sms;
  const WatchdogEnv wd = watchdog_env();
  p->timeout_ns = wd.timeout_ns;
  p->inject_stall = wd.inject_stall;
  const bool forward = epilog != GEMM_EPI_DGATED, bf16 = dtype == GEMM_EPI_BF16;
  cudaError_t e = cudaSuccess;
  if (!forward || !use_skinny(T))
    e = plan_tiles(p, bf16, forward, sms);
  else if (!plan_few(p, bf16, &e))
    e = skinny_fits(2 * N, K, sms) ? plan_skinny(p, bf16, sms) : plan_tiles(p, bf16, forward, sms);
  if (e == cudaSuccess) e = cudaHostAlloc((void**)&p->status_host, sizeof(int), cudaHostAllocMapped);
  if (e == cudaSuccess) {
    *p->status_host = 0;
    e = cudaHostGetDevicePointer((void**)&p->status_dev, p->status_host, 0);
  }
  if (e != cudaSuccess) {
    cuda_fail(e, "gated plan");
    release(p);
    return nullptr;
  }
  {
    std::lock_guard<std::mutex> lock(g_mu);
    live_plans().insert(p);
  }
  g_last_error.clear();
  return p;
}

// The weight: boxes of 64 features x a stage's k, or (N x K) of 64 k x the
// features that one load brings.
int encode_weight(CUtensorMap* map, const gemm_epi_plan_s* p, const void* W, int64_t cols, uint32_t k_rows,
                  uint32_t features) {
  if (p->w_nk) return encode_2d(map, W, (uint64_t)p->K, (uint64_t)cols, ge::kBK, features, "the N x K weight operand");
  return encode_2d(map, W, (uint64_t)cols, (uint64_t)p->K, 64, k_rows, "the weight operand");
}

int launch_tiles(gemm_epi_plan_s* p, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& y,
                 const CUtensorMap& aux, ge::TileParams& k, cudaStream_t stream) {
  k.T = (int32_t)p->T;
  k.N = (int32_t)p->N;
  k.K = (int32_t)p->K;
  k.m_tiles = p->m_tiles;
  k.n_tiles = p->n_tiles;
  k.k_blocks = p->k_blocks;
  k.num_tiles = p->num_tiles;
  k.group_m = p->group_m;
  k.raster_n = p->raster_n;
  k.status = p->status_dev;
  k.timeout_ns = p->timeout_ns;
  k.inject_stall = p->inject_stall;
  k.tail_split = p->tail_split;
  k.bias_f32 = p->bias_f32;
  k.out_f32 = p->out_f32;
  k.act = p->act;
  Launch l(p->grid, p->cfg.threads, p->cfg.smem, p->cfg.pair, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, p->cfg.fn, a, b, y, aux, k);
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "gated layer launch");
}

int run_skinny(gemm_epi_plan_s* p, const void* X, const void* W, const void* bias, void* H, void* aux,
               cudaStream_t stream) {
  CUtensorMap w, x;
  int rc = encode_weight(&w, p, W, 2 * p->N, 2 * ge::kBK, (uint32_t)p->sk_features);
  if (!rc) rc = encode_2d(&x, X, (uint64_t)p->K, (uint64_t)p->T, ge::kBK, (uint32_t)p->sk.TP, "the row operand");
  if (rc) return rc;
  ge::SkinnyParams k{};
  k.T = (int32_t)p->T;
  k.N = (int32_t)p->N;
  k.K = (int32_t)p->K;
  k.n_tiles = ceil_div(p->N, p->sk_features);
  k.kbt = p->sk_kbt;
  k.total_kb = p->sk_total;
  k.max_segs = p->sk_max_segs;
  k.bias = bias;
  k.out = H;
  k.aux_out = static_cast<uint32_t*>(aux);
  k.partials = p->sk_partials;
  k.tickets = p->sk_tickets;
  k.status = p->status_dev;
  k.timeout_ns = p->timeout_ns;
  k.bias_f32 = p->bias_f32;
  k.out_f32 = p->out_f32;
  k.cache_hints = 1;
  k.inject_stall = p->inject_stall;
  k.act = p->act;
  Launch l(p->sk_grid, ge::kThreads, p->sk.smem, false, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, p->sk.fn, w, x, k);
  if (p->inject_stall == 2) p->inject_stall = 0;
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "gated few-row launch");
}

}  // namespace

extern "C" {

gemm_epi_plan_t gemm_epi_gated_plan(int64_t T, int64_t N, int64_t K, gemm_epi_dtype dtype, gemm_epi_gated_epilog epilog,
                                    gemm_epi_act act, uint32_t flags) {
  try {
    return make_plan(T, N, K, dtype, epilog, act, flags);
  } catch (...) {  // host memory ran out
    return nullptr;
  }
}

int gemm_epi_gated_execute(gemm_epi_plan_t plan, const void* X, const void* W, const void* bias, void* H, void* aux,
                           cudaStream_t stream) {
  int rc = 0;
  gemm_epi_plan_s* p = lookup_kind(plan, 3, "gemm_epi_gated_execute", &rc);
  if (!p) return rc;
  if (p->epilog == GEMM_EPI_DGATED)
    return fail(GEMM_EPI_ERR_EPILOG_MISMATCH, "gemm_epi_gated_execute called on a DGATED plan");
  if (p->epilog != GEMM_EPI_GATED_AUX) aux = nullptr;
  if (!X || !W || !H) return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_gated_execute: NULL X, W or H");
  if (p->epilog == GEMM_EPI_GATED_AUX && !aux)
    return fail(GEMM_EPI_ERR_EPILOG_MISMATCH, "GATED_AUX needs an aux buffer");
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(H, 16) || !aligned(aux, 16) || !aligned(bias, p->bias_f32 ? 4 : 2))
    return fail(GEMM_EPI_ERR_MISALIGNED,
                "gemm_epi_gated_execute: X, W, H and aux need 16-byte, bias 2-byte (fp32: 4-byte) alignment");
  DeviceScope scope(p->device);
  rc = begin_call(p, stream);
  if (rc) return rc;
  if (p->gf.fn) return run_few(p, X, W, bias, H, aux, stream);
  if (p->kernel == 1) return run_skinny(p, X, W, bias, H, aux, stream);
  CUtensorMap a, b, y, z;
  rc = encode_2d(&a, X, (uint64_t)p->K, (uint64_t)p->T, ge::kBK, ge::kBM, "the row operand");
  if (!rc) rc = encode_weight(&b, p, W, 2 * p->N, ge::kBK, p->cfg.pair ? 64u : (uint32_t)p->cfg.BN / 2);
  if (!rc) rc = p->out_f32 ? encode_out_f32(&y, H, p->T, p->N) : encode_out(&y, H, p->T, p->N);
  if (!rc && aux) rc = encode_halves(&z, aux, p->T, p->N);
  if (rc) return rc;
  ge::TileParams k{};
  k.bias = bias;
  k.out = H;
  k.aux_out = static_cast<uint32_t*>(aux);
  return launch_tiles(p, a, b, y, aux ? z : y, k, stream);
}

int gemm_epi_dgated_execute(gemm_epi_plan_t plan, const void* dY, const void* W2, const void* aux, void* dZ, float* dbias,
                            cudaStream_t stream) {
  int rc = 0;
  gemm_epi_plan_s* p = lookup_kind(plan, 3, "gemm_epi_dgated_execute", &rc);
  if (!p) return rc;
  if (p->epilog != GEMM_EPI_DGATED)
    return fail(GEMM_EPI_ERR_EPILOG_MISMATCH, "gemm_epi_dgated_execute called on a forward plan");
  if (!dY || !W2 || !aux || !dZ) return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_dgated_execute: NULL dY, W2, aux or dZ");
  if (dbias && p->no_dbias)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_dgated_execute: dbias on a plan made with GEMM_EPI_FLAG_NO_DBIAS");
  if (!aligned(dY, 16) || !aligned(W2, 16) || !aligned(aux, 16) || !aligned(dZ, 16) || !aligned(dbias, 4))
    return fail(GEMM_EPI_ERR_MISALIGNED, "gemm_epi_dgated_execute: dY, W2, aux, dZ need 16-byte, dbias 4-byte alignment");
  DeviceScope scope(p->device);
  rc = begin_call(p, stream);
  if (rc) return rc;
  CUtensorMap a, b;
  rc = encode_2d(&a, dY, (uint64_t)p->K, (uint64_t)p->T, ge::kBK, ge::kBM, "dY");
  if (!rc) rc = encode_weight(&b, p, W2, p->N, ge::kBK, p->cfg.pair ? 64u : (uint32_t)p->cfg.BN);
  if (rc) return rc;
  ge::TileParams k{};
  k.out = dZ;
  k.aux_in = static_cast<const uint32_t*>(aux);
  k.partials = p->partials;
  k.dbias = dbias;
  rc = launch_tiles(p, a, b, a, a, k, stream);  // (outputs go out without a map)
  if (rc || !dbias) return rc;
  Launch l(ceil_div(2 * p->N, 32), 256, 0, false, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, ge::dgated_dbias_kernel, static_cast<const float*>(p->partials),
                                           ceil_div(p->T, 32), (int)(2 * p->N), dbias);
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "bias gradient launch");
}

}  // extern "C"
