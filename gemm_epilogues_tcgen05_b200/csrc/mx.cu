// mx.cu -- C ABI of the microscaled 4-bit path: quantisation, its inverse, and
// the plan and call of the product.
#include "host_common.h"
#include "mx_kernel.cuh"
#include "mx_quant.cuh"

using namespace ge_host;

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 22;  // of a row: a launch has a block row per scale tile

int64_t row_tiles(int64_t rows, int64_t groups) {
  // groups: each may end in a part of a tile
  return groups > 0 ? rows / 128 + (groups < rows ? groups : rows) : (rows + 127) / 128;
}

// the shape checks that quantisation and its inverse share
int check_shape(const char* call, int64_t batch, int64_t rows, int64_t cols, gemm_epi_dtype dtype, int64_t groups) {
  if (batch < 1 || rows < 1 || cols < 32 || cols % 32 != 0 || rows > (int64_t)1 << 30 || cols > kMaxCols ||
      batch > (int64_t)1 << 24 || batch * rows > (int64_t)1 << 36)
    return fail(GEMM_EPI_ERR_INVALID_ARG,
                "%s: bad shape batch=%lld rows=%lld cols=%lld (need all >= 1, cols a multiple of 32 and at most %lld)", call,
                (long long)batch, (long long)rows, (long long)cols, (long long)kMaxCols);
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (groups < 0 || groups > ge::kMaxExperts || (groups > 0 && batch != 1))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "%s: bad number of groups %lld (0 to %d, with one matrix)", call,
                (long long)groups, ge::kMaxExperts);
  return GEMM_EPI_OK;
}

ge::MxQuantParams quant_params(int64_t batch, int64_t rows, int64_t cols, int64_t groups, const int32_t* offsets) {
  ge::MxQuantParams k{};
  k.batch = batch;
  k.rows = rows;
  k.cols = (int32_t)cols;
  k.kt = ceil_div(cols, 128);
  k.rt = ceil_div(rows, 128);
  k.groups = (int32_t)groups;
  k.flat = batch == 1 || rows % 128 == 0;
  k.offsets = offsets;
  return k;
}

// Blocks along x for `items` of `per_block` each, `columns` blocks along y, and
// about `per_sm` blocks an SM in all.
dim3 grid_for(int64_t items, int per_block, int64_t columns, int sms, int per_sm) {
  const int64_t want = (items + per_block - 1) / per_block;
  int64_t most = ((int64_t)sms * per_sm + columns - 1) / columns;
  if (most < 1) most = 1;
  return dim3((unsigned)(want < most ? want : most), (unsigned)columns, 1);
}

size_t table_bytes(int64_t groups) { return groups > 0 ? 2 * (size_t)(groups + 1) * sizeof(int) : 0; }

int run(void (*kernel)(ge::MxQuantParams), dim3 grid, int threads, size_t smem, const ge::MxQuantParams& k,
        cudaStream_t stream) {
  Launch l(grid, threads, smem, false, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, k);
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "quantisation launch");
}

void release(gemm_epi_plan_s* p) {
  if (p->status_host) cudaFreeHost(p->status_host);
  delete p;
}

// Rows per tile, as for grouped plans: rounds of tiles x (stages of 256 k x
// time per stage + what a tile costs beside them). Measured (us, 128 / 256 rows):
// T = 4096, N = 11008, K = 4096: 137 / 74; E = 16, T = 1000, N = 5000, K = 2048:
// 21.5 / 24.1; T = 4, N = 11008, K = 4096: 8.6 / 10.2.
int choose_tr(int64_t groups, int64_t T, int64_t N, int64_t K, int sms) {
  if (const char* f = getenv("GEMM_EPI_FORCE_GROUPED")) {  // tuning override
    const int v = atoi(f);
    if (v == 128 || v == 256) return v;
  }
  const int64_t active = groups < T ? groups : T, mean = (T + active - 1) / active;
  int best = 0;
  double best_us = 0;
  for (int tr : {128, 256}) {
    const int units = tr == 256 ? sms / 2 : sms;
    const int64_t tiles = active * ((mean + tr - 1) / tr) * ((N + (tr == 256 ? 255 : 127)) / (tr == 256 ? 256 : 128));
    const double busy = tiles < units ? double(tiles) / units : 1.0;
    const double stage = tr == 256 ? (busy < 0.7 ? 0.28 : 0.4 * busy) : (busy < 0.6 ? 0.15 : 0.25 * busy);
    const double us = double((tiles + units - 1) / units) * (double((K + 255) / 256) * stage + (tr == 256 ? 1.5 : 0.8));
    if (best == 0 || us < best_us * 0.999) {
      best = tr;
      best_us = us;
    }
  }
  return best;
}

gemm_epi_plan_t make_plan(int64_t E, int64_t T, int64_t N, int64_t K, gemm_epi_dtype dtype, gemm_epi_epilog epilog,
                          uint32_t flags) {
  if ((flags & ~(uint32_t)GEMM_EPI_FLAG_OUT_F32) != 0) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown plan flags 0x%x", flags);
    return nullptr;
  }
  if (E < 0 || E > ge::kMaxExperts) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "bad number of experts %lld (need 0 to %d)", (long long)E, ge::kMaxExperts);
    return nullptr;
  }
  if (T < 1 || N < 8 || K < 32 || (N % 8) != 0 || (K % 32) != 0 || K > kMaxCols) {
    fail(GEMM_EPI_ERR_INVALID_ARG,
         "bad shape T=%lld N=%lld K=%lld (need T>=1, N a multiple of 8, K a multiple of 32 and at most %lld)", (long long)T,
         (long long)N, (long long)K, (long long)kMaxCols);
    return nullptr;
  }
  if (T > (int64_t)1 << 30 || N > (int64_t)1 << 24 || T * N > ((int64_t)1 << 40) ||
      K * N > ((int64_t)1 << 37)) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "shape too large for 32-bit tile coordinates");
    return nullptr;
  }
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    return nullptr;
  }
  if (epilog != GEMM_EPI_BIAS && epilog != GEMM_EPI_RELU_BIAS && epilog != GEMM_EPI_GELU_BIAS && epilog != GEMM_EPI_NONE) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "epilog %d has no microscaled product (BIAS, RELU_BIAS, GELU_BIAS, NONE have)",
         (int)epilog);
    return nullptr;
  }
  const int64_t groups = E > 0 ? E : 1;
  int dev = 0, sms = 0;
  if (require_b200(&dev, &sms)) return nullptr;
  const int tr = choose_tr(groups, T, N, K, sms);
  const int fm = tr == 256 ? 256 : 128;
  const int64_t n_ft = (N + fm - 1) / fm;
  const int64_t tiles = (E > 0 ? T / tr + (E < T ? E : T) : (T + tr - 1) / tr) * n_ft;
  if (tiles >= ((int64_t)1 << 31) - 65536 || groups * ((N + 127) / 128) >= ((int64_t)1 << 31) - 1) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "shape too large for 32-bit tile coordinates");
    return nullptr;
  }
  auto* p = new gemm_epi_plan_s();
  p->kind = 2;
  p->uT = p->T = T;
  p->uK = p->K = K;
  p->N = N;
  p->dtype = dtype;
  p->epilog = epilog;
  p->device = dev;
  p->num_sms = sms;
  p->out_f32 = (flags & GEMM_EPI_FLAG_OUT_F32) ? 1 : 0;
  const ge_inst::MxInstance inst = ge_inst::mx_any(tr, (int)epilog, dtype == GEMM_EPI_BF16, p->out_f32 != 0);
  GroupedCfg& g = p->gr;
  g.mx_fn = inst.fn;
  g.smem = inst.smem;
  g.threads = inst.threads;
  g.stages = inst.stages;
  g.BK = inst.bk;
  g.TR = tr;
  g.pair = tr == 256;
  g.E = (int)E;
  g.n_ft = (int)n_ft;
  p->kernel = g.pair ? 7 : 6;
  p->k_blocks = ceil_div(K, g.BK);
  const int64_t group = (int64_t)(48 << 20) / ((int64_t)tr * K / 2);  // row tiles held in L2, as in grouped plans
  g.group = (int)(group < 1 ? 1 : group > 65536 ? 65536 : group);
  const WatchdogEnv wd = watchdog_env();
  p->timeout_ns = wd.timeout_ns;
  p->inject_stall = wd.inject_stall;
  cudaError_t e = cudaFuncSetAttribute(g.mx_fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)g.smem);
  if (e == cudaSuccess) {
    if (g.pair) {
      const int pairs = resident_pairs((const void*)g.mx_fn, g.threads, g.smem, sms);
      p->grid = 2 * (int)(tiles < pairs ? tiles : pairs);
    } else {
      p->grid = (int)(tiles < sms ? tiles : sms);
    }
    e = cudaHostAlloc((void**)&p->status_host, sizeof(int), cudaHostAllocMapped);
  }
  if (e == cudaSuccess) {
    *p->status_host = 0;
    e = cudaHostGetDevicePointer((void**)&p->status_dev, p->status_host, 0);
  }
  if (e != cudaSuccess) {
    cuda_fail(e, "microscaled plan");
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

}  // namespace

extern "C" {

int64_t gemm_epi_mx_scales_bytes(int64_t batch, int64_t rows, int64_t cols, int64_t groups) {
  if (check_shape("gemm_epi_mx_scales_bytes", batch, rows, cols, GEMM_EPI_F16, groups)) return -1;
  return batch * row_tiles(rows, groups) * ((cols + 127) / 128) * 512;
}

int gemm_epi_mx_quantize(int64_t batch, int64_t rows, int64_t cols, gemm_epi_dtype dtype, uint32_t flags, const void* src,
                         const int32_t* offsets, int64_t groups, uint8_t* q, uint8_t* scales, cudaStream_t stream) {
  if (flags & ~(uint32_t)GEMM_EPI_MX_TRANSPOSED)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_mx_quantize: unknown flags 0x%x", flags);
  int rc = check_shape("gemm_epi_mx_quantize", batch, rows, cols, dtype, groups);
  if (rc) return rc;
  const bool t = (flags & GEMM_EPI_MX_TRANSPOSED) != 0;
  if (t && (rows % 8 != 0 || groups > 0))
    return fail(GEMM_EPI_ERR_INVALID_ARG,
                "gemm_epi_mx_quantize: a transposed source needs rows a multiple of 8 and no groups");
  if (!src || !q || !scales || (groups > 0 && !offsets))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_mx_quantize: NULL src, q, scales or offsets");
  if (!aligned(src, 16) || !aligned(q, 16) || !aligned(scales, 16) || (groups > 0 && !aligned(offsets, 4)))
    return fail(GEMM_EPI_ERR_MISALIGNED, "gemm_epi_mx_quantize: src, q, scales need 16-byte, offsets 4-byte alignment");
  int dev = 0, sms = 0;
  rc = require_b200(&dev, &sms);
  if (rc) return rc;
  ge::MxQuantParams k = quant_params(batch, rows, cols, groups, offsets);
  k.src = src;
  k.q = q;
  k.scales = scales;
  const bool bf16 = dtype == GEMM_EPI_BF16;
  if (t) {
    const dim3 blocks = grid_for(batch * ((rows + 63) / 64), 4, k.kt, sms, 32);
    return run(bf16 ? ge::mx_quantize_t_kernel<true> : ge::mx_quantize_t_kernel<false>, blocks, 128, 0, k, stream);
  }
  const dim3 blocks = grid_for(batch * rows, 8, (cols + 1023) / 1024, sms, 32);
  return run(bf16 ? ge::mx_quantize_kernel<true> : ge::mx_quantize_kernel<false>, blocks, 256, table_bytes(groups), k, stream);
}

int gemm_epi_mx_dequantize(int64_t batch, int64_t rows, int64_t cols, gemm_epi_dtype dtype, uint32_t flags,
                           const uint8_t* q, const uint8_t* scales, const int32_t* offsets, int64_t groups, void* out,
                           cudaStream_t stream) {
  if (flags & ~(uint32_t)GEMM_EPI_FLAG_OUT_F32)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_mx_dequantize: unknown flags 0x%x", flags);
  int rc = check_shape("gemm_epi_mx_dequantize", batch, rows, cols, dtype, groups);
  if (rc) return rc;
  if (!out || !q || !scales || (groups > 0 && !offsets))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_mx_dequantize: NULL q, scales, offsets or out");
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(scales, 16) || (groups > 0 && !aligned(offsets, 4)))
    return fail(GEMM_EPI_ERR_MISALIGNED, "gemm_epi_mx_dequantize: q, scales, out need 16-byte, offsets 4-byte alignment");
  int dev = 0, sms = 0;
  rc = require_b200(&dev, &sms);
  if (rc) return rc;
  ge::MxQuantParams k = quant_params(batch, rows, cols, groups, offsets);
  k.q = const_cast<uint8_t*>(q);
  k.scales = const_cast<uint8_t*>(scales);
  k.out = out;
  k.out_f32 = (flags & GEMM_EPI_FLAG_OUT_F32) ? 1 : 0;
  const dim3 blocks = grid_for(batch * rows, 8, (cols + 1023) / 1024, sms, 32);
  return run(dtype == GEMM_EPI_BF16 ? ge::mx_dequantize_kernel<true> : ge::mx_dequantize_kernel<false>, blocks, 256,
             table_bytes(groups), k, stream);
}

gemm_epi_plan_t gemm_epi_mx_plan(int64_t E, int64_t T, int64_t N, int64_t K, gemm_epi_dtype dtype, gemm_epi_epilog epilog,
                                 uint32_t flags) {
  try {
    return make_plan(E, T, N, K, dtype, epilog, flags);
  } catch (...) {  // host memory ran out
    return nullptr;
  }
}

int gemm_epi_mx_execute(gemm_epi_plan_t plan, const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws,
                        const void* bias, const int32_t* offsets, void* Y, cudaStream_t stream) {
  int rc = 0;
  gemm_epi_plan_s* p = lookup_kind(plan, 2, "gemm_epi_mx_execute", &rc);
  if (!p) return rc;
  const bool grouped = p->gr.E > 0;
  if (!Xq || !Xs || !Wq || !Ws || !Y || (!bias && p->epilog != GEMM_EPI_NONE) || (grouped && !offsets))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_mx_execute: NULL Xq, Xs, Wq, Ws, bias, offsets or Y");
  if (!grouped && offsets)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_mx_execute: offsets on a plan without experts");
  if (!aligned(Xq, 16) || !aligned(Xs, 16) || !aligned(Wq, 16) || !aligned(Ws, 16) || !aligned(Y, 16) ||
      !aligned(offsets, 4) || !aligned(bias, p->bias_f32 ? 4 : 2))
    return fail(GEMM_EPI_ERR_MISALIGNED,
                "gemm_epi_mx_execute: values, scales and Y need 16-byte, offsets 4-byte, bias 2-byte (fp32: 4-byte) alignment");
  DeviceScope scope(p->device);
  rc = begin_call(p, stream);
  if (rc) return rc;
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const auto plain = CU_TENSOR_MAP_SWIZZLE_NONE;
  const uint64_t N = (uint64_t)p->N, K = (uint64_t)p->K, T = (uint64_t)p->T, E = grouped ? (uint64_t)p->gr.E : 1;
  const uint64_t wt = (N + 127) / 128, kt = (K + 127) / 128;
  CUtensorMap a, b, sa, sb;
  rc = encode_3d(&a, u8, Wq, K / 2, N, E, 128, 128, "the weights");
  if (!rc) rc = encode_3d(&b, u8, Xq, K / 2, T, 1, 128, p->gr.pair ? 64 : 32, "the row operand");
  if (!rc) rc = encode_3d(&sa, u32, Ws, 128, kt, E * wt, 128, 2, "the weights' scales", plain);
  if (!rc) rc = encode_3d(&sb, u32, Xs, 128, kt, (uint64_t)row_tiles(p->T, p->gr.E), 128, 2, "the rows' scales", plain);
  if (rc) return rc;
  ge::MxParams k{};
  k.wt = (int32_t)wt;
  k.g.T = (int32_t)p->T;
  k.g.N = (int32_t)p->N;
  k.g.K = (int32_t)p->K;
  k.g.E = (int32_t)E;
  k.g.n_ft = p->gr.n_ft;
  k.g.k_blocks = p->k_blocks;
  k.g.group = p->gr.group;
  k.g.offsets = offsets;
  k.g.bias = bias;
  k.g.out = Y;
  k.g.status = p->status_dev;
  k.g.timeout_ns = p->timeout_ns;
  k.g.bias_f32 = p->bias_f32;
  k.g.out_f32 = p->out_f32;
  k.g.inject_stall = p->inject_stall;
  Launch l(p->grid, p->gr.threads, p->gr.smem, p->gr.pair, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, p->gr.mx_fn, a, b, sa, sb, k);
  if (e != cudaSuccess) return cuda_fail(e, "microscaled product launch");
  if (p->inject_stall == 2) p->inject_stall = 0;
  return GEMM_EPI_OK;
}

}  // extern "C"
