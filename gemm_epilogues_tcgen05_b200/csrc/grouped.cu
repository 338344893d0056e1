// grouped.cu -- C ABI of the products grouped by expert: plan validation and
// kernel choice, TMA descriptors, launches.
#include "grouped_kernel.cuh"
#include "host_common.h"

using namespace ge_host;

namespace {

// Rows per tile, from the mean number of rows per expert (the plan knows no
// offsets; any division of the rows is computed right by each): the least of
// rounds of tiles x time per tile. A tile of 64 k takes about 0.25 us on one
// SM while all of them load (32-row tiles less when few are busy), 0.33 us on a
// CTA pair. Measured (us, 32 / 128 / 256 rows): one expert of 1000 rows, K =
// 4096, N = 256: 12.9 / 15.3 / 23.9; four of 100, K = 2048, N = 512: 9.2 /
// 11.6 / 11.4; one of 3932, K = 192, N = 5824, DRELU_BGRAD: 334 / 47 / 27. WGRAD is
// bound by its stores where experts are short: E = 32 of
// 125 rows, K = 1024, N = 2048, fp32: 53.5 (128) and 53.8 (256); E = 8 of 1024,
// K = 4096, N = 11008: 732 and 519; E = 6 of 3, K = 3320, N = 9336: 181 and 132.
// What the mean cannot see: T = 8192 planned, 64 rows there (8 experts, K = 4096,
// N = 11008): 110 us in the plan's 256-row tiles, 112 planned for 64; T = 4096
// planned, 16 there (K = 2048, N = 512): 11.4 (128) and 9.8 (32). One expert of
// 4033 rows beside 63 of one, K = 1024, N = 4096: 129 (128, chosen) and 111 (256).
int choose_tr(int64_t E, int64_t T, int64_t N, int64_t K, int epilog, bool out_f32, int sms) {
  const bool wgrad = epilog == GEMM_EPI_WGRAD;
  if (const char* f = getenv("GEMM_EPI_FORCE_GROUPED")) {  // tuning override
    const int v = atoi(f);
    if (v == 128 || v == 256 || (v == 32 && !wgrad)) return v;
  }
  const int64_t active = E < T ? E : T, mean = (T + active - 1) / active;
  int best = 0;
  double best_us = 0;
  for (int tr : {32, 128, 256}) {
    if (wgrad && tr == 32) continue;
    const int units = tr == 256 ? sms / 2 : sms;
    const int64_t n_ft = (N + (tr == 256 ? 255 : 127)) / (tr == 256 ? 256 : 128);
    const int64_t tiles = (wgrad ? E * ((K + tr - 1) / tr) : active * ((mean + tr - 1) / tr)) * n_ft;
    const double busy = tiles < units ? double(tiles) / units : 1.0;
    const double stage = tr == 256 ? 0.33 : tr == 128 ? (busy < 0.8 ? 0.2 : 0.25 * busy) : (busy < 0.58 ? 0.145 : 0.25 * busy);
    double tile_us = double(((wgrad ? mean : K) + 63) / 64) * stage;
    // storing a tile, which the next tile's products overlap
    double store = tr == 256 ? (out_f32 ? 3.4 : 2.3) : tr == 128 ? (out_f32 ? 1.7 : 1.4) : 1.2;
    if (epilog == GEMM_EPI_DRELU_BGRAD && mean > tr) store += tr == 32 ? 6.0 : 0.6;  // joining the column sums
    if (tile_us < store) tile_us = store;
    const double us = double((tiles + units - 1) / units) * tile_us + (tr == 256 ? 4.0 : tr == 128 ? 3.0 : 2.0);
    if (best == 0 || us < best_us * 0.999) {
      best = tr;
      best_us = us;
    }
  }
  return best;
}

void release(gemm_epi_plan_s* p) {
  if (p->partials) cudaFree(p->partials);
  if (p->col_tickets) cudaFree(p->col_tickets);
  if (p->sk_partials) cudaFree(p->sk_partials);
  if (p->sk_tickets) cudaFree(p->sk_tickets);
  if (p->status_host) cudaFreeHost(p->status_host);
  delete p;
}

ge::GroupedParams params(const gemm_epi_plan_s* p, const int32_t* offsets) {
  ge::GroupedParams k{};
  k.T = (int32_t)p->uT;
  k.N = (int32_t)p->N;
  k.K = (int32_t)p->uK;
  k.E = p->gr.E;
  k.n_ft = p->gr.n_ft;
  k.n_kt = p->gr.n_kt;
  k.k_blocks = p->k_blocks;
  k.group = p->gr.group;
  k.aux_words = p->aux_words;
  k.nfb = ceil_div(p->N, 128);
  k.offsets = offsets;
  k.status = p->status_dev;
  k.timeout_ns = p->timeout_ns;
  k.bias_f32 = p->bias_f32;
  k.out_f32 = p->out_f32;
  k.inject_stall = p->inject_stall;
  k.max_items = p->split_items;
  k.force_splits = p->force_splits;
  k.split_slots = p->sk_partials;
  k.split_tickets = p->sk_tickets;
  return k;
}

int launch(gemm_epi_plan_s* p, const CUtensorMap& a, const CUtensorMap& b, const ge::GroupedParams& k,
           cudaStream_t s) {
  Launch l(p->grid, p->gr.threads, p->gr.smem, p->gr.pair, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, p->gr.fn, a, b, k);
  if (e != cudaSuccess) return cuda_fail(e, "grouped kernel launch");
  if (p->inject_stall == 2) p->inject_stall = 0;
  return GEMM_EPI_OK;
}

// the operands of a forward or DRELU_BGRAD call
int forward_maps(const gemm_epi_plan_s* p, const void* X, const void* W, CUtensorMap* a, CUtensorMap* b) {
  const auto u16 = CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const uint64_t N = (uint64_t)p->N, K = (uint64_t)p->uK, E = (uint64_t)p->gr.E;
  int rc = p->w_nk ? encode_3d(a, u16, W, K, N, E, ge::kBK, 128, "the weights")
                   : encode_3d(a, u16, W, N, K, E, 64, (uint32_t)p->gr.BK, "the weights");
  if (rc) return rc;
  const int trc = p->gr.pair ? p->gr.TR / 2 : p->gr.TR;
  return encode_3d(b, u16, X, K, (uint64_t)p->uT, 1, ge::kBK, trc < 64 ? (uint32_t)trc : 64u, "the row operand");
}

gemm_epi_plan_t make_plan(int64_t E, int64_t T, int64_t N, int64_t K, gemm_epi_dtype dtype, gemm_epi_epilog epilog,
                          uint32_t flags) {
  if ((flags & ~(uint32_t)(GEMM_EPI_FLAG_W_NK | GEMM_EPI_FLAG_OUT_F32)) != 0) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown plan flags 0x%x", flags);
    return nullptr;
  }
  const bool w_nk = (flags & GEMM_EPI_FLAG_W_NK) != 0;
  if (w_nk && epilog == GEMM_EPI_WGRAD) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "GEMM_EPI_FLAG_W_NK applies to the weight of forward and DRELU_BGRAD plans");
    return nullptr;
  }
  if (E < 1 || E > ge::kMaxExperts) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "bad number of experts %lld (need 1 to %d)", (long long)E, ge::kMaxExperts);
    return nullptr;
  }
  if (T < 1 || N < 8 || K < 8 || (N % 8) != 0 || (K % 8) != 0) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "bad shape T=%lld N=%lld K=%lld (need T>=1, N,K>=8 and multiples of 8)",
         (long long)T, (long long)N, (long long)K);
    return nullptr;
  }
  if (T > (int64_t)1 << 30 || N > (int64_t)1 << 24 || K > (int64_t)1 << 24 || T * N > ((int64_t)1 << 40) ||
      K * N > ((int64_t)1 << 37)) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "shape too large for 32-bit tile coordinates");
    return nullptr;
  }
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    return nullptr;
  }
  if (epilog < GEMM_EPI_BIAS || epilog > GEMM_EPI_GELU_AUX_BIAS) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "unknown epilog %d", (int)epilog);
    return nullptr;
  }
  const bool wgrad = epilog == GEMM_EPI_WGRAD;
  int dev = 0, sms = 0;
  if (require_b200(&dev, &sms)) return nullptr;
  const int tr = choose_tr(E, T, N, K, (int)epilog, (flags & GEMM_EPI_FLAG_OUT_F32) != 0, sms);
  const int64_t n_ft = (N + (tr == 256 ? 255 : 127)) / (tr == 256 ? 256 : 128);
  const int64_t row_tiles = T / tr + (E < T ? E : T);  // at most: every expert may end in a part of a tile
  const int64_t tiles = wgrad ? E * n_ft * ((K + tr - 1) / tr) : row_tiles * n_ft;
  if (tiles >= ((int64_t)1 << 31) - 65536) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "shape too large for 32-bit tile coordinates");
    return nullptr;
  }
  auto* p = new gemm_epi_plan_s();
  p->kind = 1;
  p->uT = p->T = T;
  p->uK = p->K = K;
  p->N = N;
  p->dtype = dtype;
  p->epilog = epilog;
  p->device = dev;
  p->num_sms = sms;
  p->w_nk = w_nk ? 1 : 0;
  p->out_f32 = (flags & GEMM_EPI_FLAG_OUT_F32) ? 1 : 0;
  p->aux_words = ceil_div(N, 32);
  const bool bf16 = dtype == GEMM_EPI_BF16;
  // Few tiles (as far as the plan can tell) with a long contraction: the
  // instance that may share a tile among CTAs, where the estimate gains at least
  // the 2 us that this instance takes longer over whole tiles (WGRAD of 2678
  // rows, K = 864, N = 208: 14.9 us, 16.6 in this instance unsplit, 15.7 in four
  // parts; forward of 2777 rows, K = 3856, N = 232: 26.4 us, 18.5 in three).
  const int64_t active = E < T ? E : T, mean = (T + active - 1) / active;
  // (WGRAD contracts over an expert's rows: one of twice the mean)
  const int64_t longest = 2 * mean < T ? 2 * mean : T;
  const int64_t stages = wgrad ? (longest + 63) / 64 : (K + (tr == 32 ? 127 : 63)) / (tr == 32 ? 128 : 64);
  const int64_t expected = wgrad ? tiles : active * ((mean + tr - 1) / tr) * n_ft;
  bool split = false;
  int parts = 1;  // with the least estimate, as the kernel would choose for these rows
  if (tr != 256 && expected <= sms) {
    const int rows = (int)(wgrad ? K : mean);
    const int64_t whole = ge::grouped_split_ns(tr, expected, 1, (int)stages, sms, rows);
    int64_t least = whole;
    for (int s = 2; s <= 16; ++s) {
      if (!ge::grouped_split_allowed(expected, s, (int)stages, sms)) continue;
      const int64_t ns = ge::grouped_split_ns(tr, expected, s, (int)stages, sms, rows);
      if (ns < least) {
        least = ns;
        parts = s;
      }
    }
    split = least + 2000 <= whole;
  }
  if (const char* f = getenv("GEMM_EPI_FORCE_SPLIT")) {  // tuning override
    p->force_splits = atoi(f) > 0 ? atoi(f) : 0;
    if (p->force_splits) {
      split = tr != 256 && p->force_splits > 1;
      const int64_t room = sms / expected;
      parts = p->force_splits < 16 ? p->force_splits : 16;
      if (parts > room) parts = room > 1 ? (int)room : 1;
    }
  }
  p->split_k = split ? parts : 1;
  const auto pick = bf16 ? (w_nk ? ge_inst::grouped_bf16_nk : ge_inst::grouped_bf16_mn)
                         : (w_nk ? ge_inst::grouped_f16_nk : ge_inst::grouped_f16_mn);
  const ge_inst::GroupedInstance inst = pick(tr, (int)epilog, split);
  GroupedCfg& g = p->gr;
  g.fn = inst.fn;
  g.smem = inst.smem;
  g.threads = inst.threads;
  g.stages = inst.stages;
  g.BK = inst.bk;
  g.TR = tr;
  g.pair = tr == 256;
  g.E = (int)E;
  g.n_ft = (int)n_ft;
  g.n_kt = ceil_div(K, tr);
  p->kernel = tr == 32 ? 3 : tr == 128 ? 4 : 5;
  p->k_blocks = ceil_div(K, g.BK);
  // row tiles whose X (about 48 MB, under half of the L2) stays in L2 while
  // the group sweeps the expert's features, each block of the weight being
  // read once per group; WGRAD holds a group of k tiles of X the same way
  const int64_t rows = wgrad ? (T + E - 1) / E : K;
  int64_t group = (int64_t)(48 << 20) / (2 * (int64_t)tr * rows);
  g.group = (int)(group < 1 ? 1 : group > 65536 ? 65536 : group);
  if (wgrad && g.group > g.n_kt) g.group = g.n_kt;
  const WatchdogEnv wd = watchdog_env();
  p->timeout_ns = wd.timeout_ns;
  p->inject_stall = wd.inject_stall;
  if (!g.fn) {
    fail(GEMM_EPI_ERR_INVALID_ARG, "no kernel instance for this epilog and layout");
    release(p);
    return nullptr;
  }
  cudaError_t e = cudaFuncSetAttribute(g.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)g.smem);
  // DRELU_BGRAD also clears dbias of experts without rows, a CTA at a time: as
  // many CTAs as that takes where the tiles are few (1000 experts, one row)
  const int64_t clearing = epilog == GEMM_EPI_DRELU_BGRAD ? E * N / 16384 : 0;
  if (e != cudaSuccess) {
    cuda_fail(e, "cudaFuncSetAttribute(max dynamic shared memory)");
    release(p);
    return nullptr;
  }
  if (g.pair) {
    const int pairs = resident_pairs((const void*)g.fn, g.threads, g.smem, sms);
    const int64_t want = tiles > clearing ? tiles : clearing;
    p->grid = 2 * (int)(want < pairs ? want : pairs);
  } else {
    const int64_t want = tiles > clearing ? tiles : clearing;
    p->grid = (int)(split || want > sms ? sms : want);  // (idle CTAs cost about 1 us)
  }
  e = cudaHostAlloc((void**)&p->status_host, sizeof(int), cudaHostAllocMapped);
  if (e != cudaSuccess) {
    cuda_fail(e, "cudaHostAlloc(status word)");
    release(p);
    return nullptr;
  }
  *p->status_host = 0;
  e = cudaHostGetDevicePointer((void**)&p->status_dev, p->status_host, 0);
  if (e == cudaSuccess && epilog == GEMM_EPI_DRELU_BGRAD) {
    if (test_hook("GEMM_EPI_INJECT_PLAN_ALLOC_FAILURE")) {
      fail(GEMM_EPI_ERR_CUDA, "injected workspace allocation failure");
      release(p);
      return nullptr;
    }
    // one row of column sums per row tile, and per expert and 128 features a
    // count of the row tiles that are in
    p->partial_bytes = (size_t)row_tiles * (size_t)N * sizeof(float);
    p->n_tickets = (int)(E * ceil_div(N, 128));
    e = cudaMalloc((void**)&p->partials, p->partial_bytes);
    if (e == cudaSuccess) e = cudaMalloc((void**)&p->col_tickets, sizeof(int) * (size_t)p->n_tickets);
    if (e == cudaSuccess) e = zero_counts(p->col_tickets, (size_t)p->n_tickets);
  }
  if (e == cudaSuccess && split) {
    p->split_items = sms;  // one work item an SM: more parts never paid
    p->split_bytes = (size_t)p->split_items * tr * 128 * sizeof(float) + sizeof(int) * (size_t)p->split_items;
    e = cudaMalloc((void**)&p->sk_partials, (size_t)p->split_items * tr * 128 * sizeof(float));
    if (e == cudaSuccess) e = cudaMalloc((void**)&p->sk_tickets, sizeof(int) * (size_t)p->split_items);
    if (e == cudaSuccess) e = zero_counts(p->sk_tickets, (size_t)p->split_items);
  }
  if (e == cudaSuccess && wgrad) {
    // the optional bias gradient: row slices for about eight blocks an SM (one
    // expert may hold all the rows: E = 32, K = 1024, 4000 rows, 631 of them in
    // one expert, took 18.5 us with two slices)
    const int64_t blocks = E * ceil_div(K, 256);
    int64_t s = 8 * (int64_t)sms / blocks;
    const int64_t most = (T + 63) / 64;
    s = s > most ? most : s;
    g.slices = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
    if (g.slices > 1) {
      p->partial_bytes = (size_t)g.slices * (size_t)E * (size_t)K * sizeof(float);
      p->n_tickets = (int)blocks;
      e = cudaMalloc((void**)&p->partials, p->partial_bytes);
      if (e == cudaSuccess) e = cudaMalloc((void**)&p->col_tickets, sizeof(int) * (size_t)p->n_tickets);
      if (e == cudaSuccess) e = zero_counts(p->col_tickets, (size_t)p->n_tickets);
    }
  }
  if (e != cudaSuccess) {
    cuda_fail(e, "grouped plan workspace");
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

gemm_epi_plan_t gemm_epi_grouped_plan(int64_t E, int64_t T, int64_t N, int64_t K, gemm_epi_dtype dtype,
                                      gemm_epi_epilog epilog, uint32_t flags) {
  try {
    return make_plan(E, T, N, K, dtype, epilog, flags);
  } catch (...) {  // host memory ran out
    return nullptr;
  }
}

int gemm_epi_grouped_execute(gemm_epi_plan_t plan, const void* X, const void* W, const void* bias,
                             const int32_t* offsets, void* Y, uint32_t* aux, cudaStream_t stream) {
  int rc = 0;
  gemm_epi_plan_s* p = lookup_kind(plan, 1, "gemm_epi_grouped_execute", &rc);
  if (!p) return rc;
  if (p->epilog == GEMM_EPI_DRELU_BGRAD || p->epilog == GEMM_EPI_WGRAD)
    return fail(GEMM_EPI_ERR_EPILOG_MISMATCH, "gemm_epi_grouped_execute called on a %s plan",
                p->epilog == GEMM_EPI_WGRAD ? "WGRAD" : "DRELU_BGRAD");
  if (!X || !W || !Y || !offsets || (!bias && p->epilog != GEMM_EPI_NONE))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_grouped_execute: NULL X, W, bias, offsets or Y");
  const bool gelu_aux = p->epilog == GEMM_EPI_GELU_AUX_BIAS;
  if ((p->epilog == GEMM_EPI_RELU_AUX_BIAS || gelu_aux) && !aux)
    return fail(GEMM_EPI_ERR_EPILOG_MISMATCH, "%s needs an aux buffer", gelu_aux ? "GELU_AUX_BIAS" : "RELU_AUX_BIAS");
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(offsets, 4) ||
      !aligned(bias, p->bias_f32 ? 4 : 2) || (p->epilog == GEMM_EPI_RELU_AUX_BIAS && !aligned(aux, 4)) ||
      (gelu_aux && !aligned(aux, 16)))
    return fail(GEMM_EPI_ERR_MISALIGNED,
                "gemm_epi_grouped_execute: X, W, Y need 16-byte, offsets and aux 4-byte (GELU_AUX_BIAS: 16-byte), bias "
                "2-byte (fp32: 4-byte) alignment");
  DeviceScope scope(p->device);
  rc = begin_call(p, stream);
  if (rc) return rc;
  CUtensorMap a, b;
  rc = forward_maps(p, X, W, &a, &b);
  if (rc) return rc;
  ge::GroupedParams k = params(p, offsets);
  k.bias = bias;
  k.out = Y;
  k.aux_out = aux;
  return launch(p, a, b, k, stream);
}

int gemm_epi_grouped_drelu_bgrad_execute(gemm_epi_plan_t plan, const void* dY2, const void* W2, const uint32_t* aux,
                                         const int32_t* offsets, void* dZ, float* dbias, cudaStream_t stream) {
  int rc = 0;
  gemm_epi_plan_s* p = lookup_kind(plan, 1, "gemm_epi_grouped_drelu_bgrad_execute", &rc);
  if (!p) return rc;
  if (p->epilog != GEMM_EPI_DRELU_BGRAD)
    return fail(GEMM_EPI_ERR_EPILOG_MISMATCH,
                "gemm_epi_grouped_drelu_bgrad_execute called on a plan whose epilog is not DRELU_BGRAD");
  if (!dY2 || !W2 || !aux || !offsets || !dZ || !dbias)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_grouped_drelu_bgrad_execute: NULL dY2, W2, aux, offsets, dZ or dbias");
  if (!aligned(dY2, 16) || !aligned(W2, 16) || !aligned(dZ, 16) || !aligned(aux, 4) || !aligned(offsets, 4) ||
      !aligned(dbias, 4))
    return fail(GEMM_EPI_ERR_MISALIGNED,
                "gemm_epi_grouped_drelu_bgrad_execute: dY2, W2, dZ need 16-byte, aux, offsets, dbias 4-byte alignment");
  DeviceScope scope(p->device);
  rc = begin_call(p, stream);
  if (rc) return rc;
  CUtensorMap a, b;
  rc = forward_maps(p, dY2, W2, &a, &b);
  if (rc) return rc;
  ge::GroupedParams k = params(p, offsets);
  k.out = dZ;
  k.aux_in = aux;
  k.dbias = dbias;
  k.partials = p->partials;
  k.tickets = p->col_tickets;
  return launch(p, a, b, k, stream);
}

int gemm_epi_grouped_wgrad_execute(gemm_epi_plan_t plan, const void* X, const void* dZ, const int32_t* offsets, void* dW,
                                   float* dbias, cudaStream_t stream) {
  int rc = 0;
  gemm_epi_plan_s* p = lookup_kind(plan, 1, "gemm_epi_grouped_wgrad_execute", &rc);
  if (!p) return rc;
  if (p->epilog != GEMM_EPI_WGRAD)
    return fail(GEMM_EPI_ERR_EPILOG_MISMATCH, "gemm_epi_grouped_wgrad_execute called on a plan whose epilog is not WGRAD");
  if (!X || !dZ || !offsets || !dW)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "gemm_epi_grouped_wgrad_execute: NULL X, dZ, offsets or dW");
  if (!aligned(X, 16) || !aligned(dZ, 16) || !aligned(dW, 16) || !aligned(offsets, 4) || (dbias && !aligned(dbias, 4)))
    return fail(GEMM_EPI_ERR_MISALIGNED,
                "gemm_epi_grouped_wgrad_execute: X, dZ, dW need 16-byte, offsets and dbias 4-byte alignment");
  DeviceScope scope(p->device);
  rc = begin_call(p, stream);
  if (rc) return rc;
  const auto u16 = CU_TENSOR_MAP_DATA_TYPE_UINT16;
  CUtensorMap a, b;
  rc = encode_3d(&a, u16, dZ, (uint64_t)p->N, (uint64_t)p->uT, 1, 64, ge::kBK, "dZ");
  if (rc) return rc;
  rc = encode_3d(&b, u16, X, (uint64_t)p->uK, (uint64_t)p->uT, 1, 64, ge::kBK, "X");
  if (rc) return rc;
  ge::GroupedParams k = params(p, offsets);
  k.out = dW;
  rc = launch(p, a, b, k, stream);
  if (rc || !dbias) return rc;
  const dim3 grid((unsigned)ceil_div(p->uK, 256), (unsigned)p->gr.E, (unsigned)p->gr.slices);
  const auto kernel = p->dtype == GEMM_EPI_BF16 ? ge::grouped_colsum_kernel<true> : ge::grouped_colsum_kernel<false>;
  Launch l(grid, 256, 0, false, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, (const uint16_t*)X, offsets, (int)p->uT, p->gr.E, (int)p->uK,
                                           p->gr.slices, p->partials, p->col_tickets, dbias);
  if (e != cudaSuccess) return cuda_fail(e, "grouped bias-gradient launch");
  return GEMM_EPI_OK;
}

}  // extern "C"
