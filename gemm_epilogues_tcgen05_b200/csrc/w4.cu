// w4.cu -- C ABI of 4-bit weights with group scales: quantisation, packing, the
// inverse, and the plan and call of the product with few rows.
#include "host_tiles.h"
#include "w4_few.cuh"
#include "w4_quant.cuh"

using namespace ge_host;

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 22;
constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int kMaxT = 256;

int64_t row_tiles(int64_t rows) { return (rows + 31) / 32; }
int64_t col_tiles(int64_t cols) { return (cols + 127) / 128; }

int check_shape(const char* call, int64_t batch, int64_t rows, int64_t cols, int64_t group) {
  if (group != 32 && group != 64 && group != 128)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "%s: bad group %lld (32, 64 or 128)", call, (long long)group);
  if (batch < 1 || rows < 1 || cols < group || cols % group != 0 || rows > kMaxRows || cols > kMaxCols ||
      batch > (int64_t)1 << 20 || batch * row_tiles(rows) * col_tiles(cols) > (int64_t)1 << 40)
    return fail(GEMM_EPI_ERR_INVALID_ARG,
                "%s: bad shape batch=%lld rows=%lld cols=%lld (need all >= 1, cols a multiple of the group and at most %lld)",
                call, (long long)batch, (long long)rows, (long long)cols, (long long)kMaxCols);
  return GEMM_EPI_OK;
}

int check_dtype(gemm_epi_dtype dtype) {
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  return GEMM_EPI_OK;
}

ge::W4Params base_params(int64_t batch, int64_t rows, int64_t cols, int64_t group) {
  ge::W4Params k{};
  k.rows = (int32_t)rows;
  k.cols = (int32_t)cols;
  k.rt = (int32_t)row_tiles(rows);
  k.kt = (int32_t)col_tiles(cols);
  k.tiles = batch * k.rt * k.kt;
  k.group = (int32_t)group;
  return k;
}

// two tiles side by side a CTA (2^31 of them would be more memory than there is)
int64_t pair_blocks(const ge::W4Params& k, int64_t batch) { return batch * k.rt * ((k.kt + 1) / 2); }

// a warp takes a tile, at most 32 CTAs an SM
int64_t tile_blocks(const ge::W4Params& k, int sms) {
  const int64_t want = (k.tiles + 7) / 8, most = (int64_t)sms * 32;
  return want < most ? want : most;
}

int run(void (*kernel)(ge::W4Params), const ge::W4Params& k, int64_t blocks, cudaStream_t stream) {
  if (blocks >= (int64_t)1 << 31) return fail(GEMM_EPI_ERR_INVALID_ARG, "too many tiles for one launch");
  Launch l((int)blocks, 256, 0, false, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, k);
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "4-bit weight launch");
}

// The kernel whose warps do everything alone (w4_few.cuh), 16 rows at most a CTA: clusters along
// the features, the CTAs of one along the columns. What a launch takes goes by
// the half tiles of a warp; a join over a cluster costs about what four take. False: a
// plan on tensor memory (w4_kernel.cuh) is the faster one.
// Rows beyond 16 are another pass over the weight here, and a slower stage there, whose
// launches take 9 to 16 us before the first of them. bf16, us here / there, G = 128 | G = 32 with zeros | gated, G = 128 |
// gated, G = 32 with zeros:
//   half tiles of a warp   8: T = 32, K = N = 4096             10.1 / 15.4 | 11.7 / 16.3 | 16.0 / 26.8 | 18.6 / 29.5
//                         14: T = 64, K = N = 4096             16.4 / 18.1 | 18.6 / 19.8 | 24.7 / 30.6 | 28.5 / 35.6
//                         16: T = 48, K = 4096, N = 6144       17.3 / 17.8 | 19.9 / 24.2 | 26.9 / 28.7 | 29.9 / 43.0
//                         19: T = 64, K = 2048, N = 11008      22.3 / 18.7 | 26.5 / 25.4 | 34.6 / 30.2 | 39.5 / 42.7
//                         20: T = 32, K = 4096, N = 11008      21.1 / 19.2 | 23.5 / 23.3 | 31.9 / 32.8 | 38.0 / 41.7
//                         22: T = 48, K = 4096, N = 8192       24.3 / 19.7 | 27.6 / 28.2 | 36.3 / 33.9 | 41.4 / 51.6
//                         30: T = 48, K = 4096, N = 11008      30.4 / 22.0 | 34.0 / 36.4 | 46.8 / 38.9 | 53.5 / 65.8
// so up to 16 of a plain product and 20 of a gated one (G = 64: 19 23.2 / 19.2, gated 20 32.7 / 34.2, 22 37.6 / 39.3).
// Up to 16 rows always: T = 16, K = 4096, N = 11008 14.7 / 16.4, gated 21.2 / 27.1.
bool plan_few(gemm_epi_plan_s* p, bool gated, int64_t group, cudaError_t* e) {
  bool forced = false;
  if (const char* f = getenv("GEMM_EPI_FORCE_KERNEL")) {  // tuning override
    if (!strcmp(f, "tmem")) return false;
    forced = !strcmp(f, "warp");
  }
  // (the grid of the other kernel; a stall needs a wait)
  if (!forced && (getenv("GEMM_EPI_SKINNY_GRID") || p->inject_stall)) return false;
  W4Cfg& c = p->w4;
  c.few = (p->dtype == GEMM_EPI_BF16 ? ge_inst::w4_few_bf16 : ge_inst::w4_few_f16)((int)p->T, gated, (int)(128 / group));
  for (int z = 0; z < 2 && *e == cudaSuccess; ++z)
    *e = cudaFuncSetAttribute(c.few.fn[z], cudaFuncAttributeMaxDynamicSharedMemorySize, (int)c.few.smem[z]);
  if (*e != cudaSuccess) return true;
  c.stages = c.few.stages;
  c.tp = p->T <= 8 ? 8 : 16;
  c.row_blocks = ceil_div(p->T, c.tp);
  const FewChoice choice =
      choose_few((const void*)c.few.fn[0], c.few.threads, c.few.smem[0], p->N, c.kt, p->num_sms, c.row_blocks, 4);
  if (p->T > 16 && !forced && choice.steps > (gated ? 20 : 16)) {
    c.few = {};
    return false;
  }
  c.few_split = few_split(choice, p->N, c.kt);
  c.grid = choice.clusters << choice.split;
  p->grid = c.grid * c.row_blocks;
  c.max_segs = 1 << choice.split;
  return true;
}

// The kernel of many warps' roles (w4_kernel.cuh).
cudaError_t plan_tmem(gemm_epi_plan_s* p, bool gated, int64_t group) {
  W4Cfg& c = p->w4;
  const int most = gated && group == 128 ? 64 : (int)group;  // rows of an instance
  c.tp = p->T <= 16 ? 16 : p->T <= 32 ? 32 : p->T <= 64 ? 64 : 128;
  if (c.tp > most) c.tp = most;
  c.row_blocks = ceil_div(p->T, c.tp);
  const ge_inst::W4Instance inst = (p->dtype == GEMM_EPI_BF16 ? ge_inst::w4_bf16 : ge_inst::w4_f16)(c.tp, gated, (int)(128 / group));
  c.fn = inst.fn;
  c.smem = inst.smem;
  c.threads = inst.threads;
  c.stages = inst.stages;
  // equal shares of all blocks of 128 columns, at least two each
  const int total = c.tiles * c.kt, share = p->num_sms > c.row_blocks ? p->num_sms / c.row_blocks : 1;
  c.grid = total / 2 < 1 ? 1 : total / 2 < share ? total / 2 : share;
  if (const char* f = getenv("GEMM_EPI_SKINNY_GRID")) {  // tuning override
    const int v = atoi(f);
    if (v >= 1 && v <= total && v <= share) c.grid = v;
  }
  p->grid = c.grid * c.row_blocks;
  for (int t = 0; t < c.tiles; ++t) {
    const int64_t first = ge::skinny_owner((int64_t)t * c.kt, c.grid, total);
    const int64_t last = ge::skinny_owner((int64_t)(t + 1) * c.kt - 1, c.grid, total);
    if (last - first + 1 > c.max_segs) c.max_segs = (int)(last - first + 1);
  }
  cudaError_t e = cudaFuncSetAttribute(c.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)c.smem);
  if (e == cudaSuccess && c.max_segs > 1) {
    const size_t blocks = (size_t)c.row_blocks * (size_t)c.tiles, items = blocks * (size_t)inst.tickets;
    p->sk_bytes = blocks * (size_t)c.max_segs * (gated ? 2 : 1) * (size_t)c.tp * 128 * sizeof(float);
    e = cudaMalloc((void**)&p->sk_partials, p->sk_bytes);
    if (e == cudaSuccess) e = cudaMalloc((void**)&p->sk_tickets, sizeof(int) * items);
    if (e == cudaSuccess) e = zero_counts(p->sk_tickets, items);
    p->split_items = (int)items;
    p->sk_bytes += sizeof(int) * items;
  }
  return e;
}

gemm_epi_plan_t make_plan(int64_t T, int64_t N, int64_t K, int64_t group, gemm_epi_dtype dtype, int epilog,
                          gemm_epi_act act, uint32_t flags) {
  if ((flags & ~(uint32_t)GEMM_EPI_FLAG_OUT_F32) != 0) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown plan flags 0x%x", flags);
    return nullptr;
  }
  if (T < 1 || T > kMaxT || N < 8 || N % 8 != 0) {
    fail(GEMM_EPI_ERR_INVALID_ARG,
         "bad shape T=%lld N=%lld (need 1 <= T <= %d -- for more rows gemm_epi_w4_dequantize and a plan with "
         "GEMM_EPI_FLAG_W_NK -- and N a multiple of 8)",
         (long long)T, (long long)N, kMaxT);
    return nullptr;
  }
  const bool gated = epilog == GEMM_EPI_GATED;
  if (check_shape("gemm_epi_w4_plan", gated ? 2 : 1, N, K, group) || check_dtype(dtype)) return nullptr;
  if (!gated && epilog != GEMM_EPI_BIAS && epilog != GEMM_EPI_RELU_BIAS && epilog != GEMM_EPI_GELU_BIAS &&
      epilog != GEMM_EPI_NONE) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "epilog %d has no product with 4-bit weights (BIAS, RELU_BIAS, GELU_BIAS, NONE, GATED have)",
         epilog);
    return nullptr;
  }
  if (act != GEMM_EPI_SILU && act != GEMM_EPI_GELU && act != GEMM_EPI_RELU) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    return nullptr;
  }
  int dev = 0, sms = 0;
  if (require_b200(&dev, &sms)) return nullptr;
  const int64_t tiles = (N + 127) / 128, kt = col_tiles(K);
  if ((tiles * kt + 1) * sms >= (int64_t)1 << 31) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "shape too large for 32-bit tile coordinates");
    return nullptr;
  }
  auto* p = new gemm_epi_plan_s();
  p->kind = 4;
  p->kernel = 8;
  p->uT = p->T = T;
  p->uK = p->K = K;
  p->N = N;
  p->dtype = dtype;
  p->epilog = epilog;
  p->act = act;
  p->out_f32 = (flags & GEMM_EPI_FLAG_OUT_F32) ? 1 : 0;
  p->device = dev;
  p->num_sms = sms;
  const WatchdogEnv wd = watchdog_env();
  p->timeout_ns = wd.timeout_ns;
  p->inject_stall = wd.inject_stall;
  W4Cfg& c = p->w4;
  c.tiles = (int)tiles;
  c.kt = (int)kt;
  cudaError_t e = cudaSuccess;
  if (!plan_few(p, gated, group, &e)) e = plan_tmem(p, gated, group);
  if (e == cudaSuccess) e = cudaHostAlloc((void**)&p->status_host, sizeof(int), cudaHostAllocMapped);
  if (e == cudaSuccess) {
    *p->status_host = 0;
    e = cudaHostGetDevicePointer((void**)&p->status_dev, p->status_host, 0);
  }
  if (e != cudaSuccess) {
    cuda_fail(e, "plan of 4-bit weights");
    if (p->sk_partials) cudaFree(p->sk_partials);
    if (p->sk_tickets) cudaFree(p->sk_tickets);
    if (p->status_host) cudaFreeHost(p->status_host);
    delete p;
    return nullptr;
  }
  {
    std::lock_guard<std::mutex> lock(g_mu);
    live_plans().insert(p);
  }
  g_last_error.clear();
  return p;
}

}  // namespace

extern "C" {

int64_t gemm_epi_w4_bytes(int64_t batch, int64_t rows, int64_t cols, int64_t group) {
  if (check_shape("gemm_epi_w4_bytes", batch, rows, cols, group)) return -1;
  return batch * row_tiles(rows) * col_tiles(cols) * 2048;
}

int64_t gemm_epi_w4_scales(int64_t batch, int64_t rows, int64_t cols, int64_t group) {
  if (check_shape("gemm_epi_w4_scales", batch, rows, cols, group)) return -1;
  return batch * row_tiles(rows) * col_tiles(cols) * 32 * (128 / group);
}

int gemm_epi_w4_quantize(int64_t batch, int64_t rows, int64_t cols, int64_t group, gemm_epi_dtype dtype, const void* W,
                         uint8_t* q, void* scales, uint8_t* zeros, cudaStream_t stream) {
  int rc = check_shape("gemm_epi_w4_quantize", batch, rows, cols, group);
  if (!rc) rc = check_dtype(dtype);
  if (rc) return rc;
  if (!W || !q || !scales) return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_w4_quantize: NULL W, q or scales");
  if (!aligned(W, 16) || !aligned(q, 16) || !aligned(scales, 16) || !aligned(zeros, 16))
    return fail(GEMM_EPI_ERR_MISALIGNED, "gemm_epi_w4_quantize: W, q, scales and zeros need 16-byte alignment");
  int dev = 0, sms = 0;
  rc = require_b200(&dev, &sms);
  if (rc) return rc;
  ge::W4Params k = base_params(batch, rows, cols, group);
  k.src = W;
  k.q = q;
  k.scales = scales;
  k.zeros = zeros;
  const int64_t blocks = pair_blocks(k, batch);
  if (dtype == GEMM_EPI_BF16)
    return run(zeros ? ge::w4_quantize_kernel<true, true> : ge::w4_quantize_kernel<true, false>, k, blocks, stream);
  return run(zeros ? ge::w4_quantize_kernel<false, true> : ge::w4_quantize_kernel<false, false>, k, blocks, stream);
}

int gemm_epi_w4_pack(int64_t batch, int64_t rows, int64_t cols, int64_t group, const uint8_t* codes,
                     const void* src_scales, const uint8_t* src_zeros, uint8_t* q, void* scales, uint8_t* zeros,
                     cudaStream_t stream) {
  int rc = check_shape("gemm_epi_w4_pack", batch, rows, cols, group);
  if (rc) return rc;
  if (!codes || !src_scales || !q || !scales || (src_zeros == nullptr) != (zeros == nullptr))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_w4_pack: NULL codes, scales or q, or zeros on one side alone");
  if (!aligned(codes, 16) || !aligned(src_scales, 2) || !aligned(q, 16) || !aligned(scales, 16) || !aligned(zeros, 16))
    return fail(GEMM_EPI_ERR_MISALIGNED,
                "gemm_epi_w4_pack: codes, q, scales and zeros need 16-byte, the given scales 2-byte alignment");
  int dev = 0, sms = 0;
  rc = require_b200(&dev, &sms);
  if (rc) return rc;
  ge::W4Params k = base_params(batch, rows, cols, group);
  k.src = codes;
  k.src_scales = src_scales;
  k.src_zeros = src_zeros;
  k.q = q;
  k.scales = scales;
  k.zeros = zeros;
  return run(ge::w4_pack_kernel, k, tile_blocks(k, sms), stream);
}

int gemm_epi_w4_dequantize(int64_t batch, int64_t rows, int64_t cols, int64_t group, gemm_epi_dtype dtype, uint32_t flags,
                           const uint8_t* q, const void* scales, const uint8_t* zeros, void* out, cudaStream_t stream) {
  if (flags & ~(uint32_t)GEMM_EPI_FLAG_OUT_F32)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_w4_dequantize: unknown flags 0x%x", flags);
  int rc = check_shape("gemm_epi_w4_dequantize", batch, rows, cols, group);
  if (!rc) rc = check_dtype(dtype);
  if (rc) return rc;
  if (!q || !scales || !out) return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_w4_dequantize: NULL q, scales or out");
  if (!aligned(q, 16) || !aligned(scales, 16) || !aligned(zeros, 16) || !aligned(out, 16))
    return fail(GEMM_EPI_ERR_MISALIGNED, "gemm_epi_w4_dequantize: q, scales, zeros and out need 16-byte alignment");
  int dev = 0, sms = 0;
  rc = require_b200(&dev, &sms);
  if (rc) return rc;
  ge::W4Params k = base_params(batch, rows, cols, group);
  k.q = const_cast<uint8_t*>(q);
  k.scales = const_cast<void*>(scales);
  k.zeros = const_cast<uint8_t*>(zeros);
  k.out = out;
  const bool f32 = (flags & GEMM_EPI_FLAG_OUT_F32) != 0;
  if (dtype == GEMM_EPI_BF16)
    return run(f32 ? ge::w4_dequantize_kernel<true, true> : ge::w4_dequantize_kernel<true, false>, k, pair_blocks(k, batch), stream);
  return run(f32 ? ge::w4_dequantize_kernel<false, true> : ge::w4_dequantize_kernel<false, false>, k, pair_blocks(k, batch), stream);
}

gemm_epi_plan_t gemm_epi_w4_plan(int64_t T, int64_t N, int64_t K, int64_t group, gemm_epi_dtype dtype, int epilog,
                                 gemm_epi_act act, uint32_t flags) {
  try {
    return make_plan(T, N, K, group, dtype, epilog, act, flags);
  } catch (...) {  // host memory ran out
    return nullptr;
  }
}

int gemm_epi_w4_execute(gemm_epi_plan_t plan, const void* X, const uint8_t* q, const void* scales, const uint8_t* zeros,
                        const void* bias, void* Y, cudaStream_t stream) {
  int rc = 0;
  gemm_epi_plan_s* p = lookup_kind(plan, 4, "gemm_epi_w4_execute", &rc);
  if (!p) return rc;
  const bool optional_bias = p->epilog == GEMM_EPI_NONE || p->epilog == GEMM_EPI_GATED;
  if (!X || !q || !scales || !Y || (!bias && !optional_bias))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_w4_execute: NULL X, q, scales, bias or Y");
  if (!aligned(X, 16) || !aligned(q, 16) || !aligned(scales, 16) || !aligned(zeros, 16) || !aligned(Y, 16) ||
      !aligned(bias, p->bias_f32 ? 4 : 2))
    return fail(GEMM_EPI_ERR_MISALIGNED,
                "gemm_epi_w4_execute: X, q, scales, zeros and Y need 16-byte, bias 2-byte (fp32: 4-byte) alignment");
  DeviceScope scope(p->device);
  rc = begin_call(p, stream);
  if (rc) return rc;
  const W4Cfg& c = p->w4;
  ge::W4MulParams k{};
  k.T = (int32_t)p->T;
  k.N = (int32_t)p->N;
  k.K = (int32_t)p->K;
  k.rt = (int32_t)row_tiles(p->N);
  k.kt = c.kt;
  k.total = c.tiles * c.kt;
  k.max_segs = c.max_segs;
  k.epi = p->epilog;
  k.act = p->act;
  k.bias_f32 = p->bias_f32;
  k.out_f32 = p->out_f32;
  k.q = q;
  k.scales = scales;
  k.zeros = zeros;
  k.bias = p->epilog == GEMM_EPI_NONE ? nullptr : bias;
  k.out = Y;
  k.partials = p->sk_partials;
  k.tickets = p->sk_tickets;
  k.status = p->status_dev;
  k.timeout_ns = p->timeout_ns;
  k.inject_stall = p->inject_stall;
  if (c.few.threads) {
    k.few = c.few_split;
    k.X = X;
    Launch l(dim3((unsigned)c.grid, (unsigned)c.row_blocks, 1), c.few.threads, c.few.smem[zeros != nullptr], c.few_split.split > 0, stream);
    l.attr[1].val.clusterDim.x = 1u << c.few_split.split;
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, c.few.fn[zeros != nullptr], k);
    return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "launch of the product with 4-bit weights");
  }
  CUtensorMap x;
  rc = encode_2d(&x, X, (uint64_t)p->K, (uint64_t)p->T, ge::kBK, (uint32_t)c.tp, "the row operand");
  if (rc) return rc;
  Launch l(dim3((unsigned)c.grid, (unsigned)c.row_blocks, 1), c.threads, c.smem, false, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, c.fn, x, k);
  if (p->inject_stall == 2) p->inject_stall = 0;
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "launch of the product with 4-bit weights");
}

}  // extern "C"
