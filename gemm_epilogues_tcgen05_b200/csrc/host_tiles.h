// host_tiles.h -- what the dense and the gated plans share on the host: the
// tensor maps of 16-bit operands and of the tile kernels' outputs, the cost
// model behind the choice of tiles, and the tile order.
#pragma once

#include "host_common.h"
#include "tile_kernel.cuh"

namespace ge_host {

// 2-D row-major tensor of 16-bit elements: `inner` contiguous columns,
// `outer` rows; box of box_inner x box_outer with 128-byte swizzle (operand
// tiles) or 64-byte swizzle (32 x 32 output staging blocks).
inline int encode_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                     uint32_t box_outer, const char* name,
                     CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(GEMM_EPI_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (inject_encode_failure()) return fail(GEMM_EPI_ERR_CUDA, "injected tensor map encode failure");
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {inner * 2};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(GEMM_EPI_ERR_CUDA, "tensor map encode for %s failed (CUresult %d)", name, (int)r);
  return GEMM_EPI_OK;
}

// the output (Y, dZ or an unfused intermediate) as the tile kernels' TMA
// stores see it: 32 x 32 blocks, 64-byte swizzle
inline int encode_out(CUtensorMap* map, const void* out, int64_t T, int64_t N) {
  return encode_2d(map, out, (uint64_t)N, (uint64_t)T, 32, 32, "the output", CU_TENSOR_MAP_SWIZZLE_64B);
}

// fp32 output: 16 x 32 blocks (64-byte rows, the 16-bit blocks' staging layout)
inline int encode_out_f32(CUtensorMap* map, const void* out, int64_t T, int64_t N) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(GEMM_EPI_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (inject_encode_failure()) return fail(GEMM_EPI_ERR_CUDA, "injected tensor map encode failure");
  const cuuint64_t dims[2] = {(uint64_t)N, (uint64_t)T};
  const cuuint64_t strides[1] = {(uint64_t)N * 4};
  const cuuint32_t box[2] = {16, 32};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(out), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(GEMM_EPI_ERR_CUDA, "tensor map encode for the fp32 output failed (CUresult %d)", (int)r);
  return GEMM_EPI_OK;
}

// Kernel and tile choice by a small cost model, fitted to measurements on
// one B200 (bf16, K = 4096, one tile per CTA, events around each call):
// the one-CTA kernel's throughput per SM grows with the tile width, because
// every stage brings the same 16 KB of X for BN/64 times the MMA work --
// about 3.1, 5.4, 7.5 and 9.3 TFLOP/s per SM at BN = 64, 128, 192 and 256
// (e.g. T = 512, N = K = 4096: 49.1 us with 256 tiles of BN = 64, 30.7 us
// with 128 of BN = 128). CTA pairs (256 x 256 tiles, two thirds of the
// operand bytes per FLOP) run about 10 per SM. A plan's estimate is rounds
// of tiles x time per tile; the pair kernel's last round counts half when its
// tiles fit the half-width tail split.
inline double tile_rate(int bn) { return bn == 256 ? 9.3 : bn == 192 ? 7.5 : bn == 128 ? 5.4 : 3.1; }
constexpr double kPairRate = 10.0;

inline double est_tile_us(int64_t T, int64_t N, int64_t K, int bn, int sms) {
  const int64_t tiles = ((T + ge::kBM - 1) / ge::kBM) * ((N + bn - 1) / bn);
  const int64_t rounds = (tiles + sms - 1) / sms;
  return double(rounds) * 2.0 * ge::kBM * bn * double(K) / (tile_rate(bn) * 1e6);
}

inline double est_pair_us(int64_t T, int64_t N, int64_t K, int pairs) {
  const int64_t tiles = ((T + 255) / 256) * ((N + 255) / 256);
  const int64_t full = tiles / pairs, tail = tiles % pairs;
  const double rounds = double(full) + (tail == 0 ? 0.0 : 2 * tail <= pairs ? 0.5 : 1.0);
  return rounds * 2.0 * 256 * 256 * double(K) / (2.0 * kPairRate * 1e6);
}

// The few-row kernel's range arithmetic is 32-bit: (k-blocks + 1) x grid must
// stay below 2^31 (k-blocks of 64 at most, grid at most one CTA per SM).
inline bool skinny_fits(int64_t N, int64_t K, int sms) {
  const int64_t kblocks = ((N + 127) / 128) * ((K + 63) / 64);
  return (kblocks + 1) * (int64_t)sms < (int64_t(1) << 31);
}

// Raster: which operand's block stays in L2 while the other streams past
// it. Holding a group of R row tiles of X (about 48 MB, a little under half
// of the 126 MB L2) while the group sweeps every column block streams W from
// HBM once per group -- once in all when all of X fits (FFN, square). When X
// is both larger than the L2 and at least 4x W, a group of column tiles of W
// (about 64 MB) is held instead and X streams past it. Measured on the
// 65536 x 16384 x 8192 fp16 problem (X 2 GiB, W 256 MiB; ncu, DRAM bytes read
// per launch, one-CTA kernel, 256-column tiles): row groups 24.3 GB; column
// groups of 6, 8 and 12 tiles 20.1, 18.0 and 19.2 GB, at equal time (13.4 to
// 13.8 ms). Every order reads several times the operands there: a wave of
// 148 tiles touches 1.8 GB of operands at K = 16384, 14 times the L2.
// GEMM_EPI_RASTER=m|n and GEMM_EPI_GROUP_M (the group size in tiles)
// override, for measurement.
struct Raster {
  int group = 1;
  int by_n = 0;
};

inline Raster choose_raster(int64_t T, int64_t N, int64_t K, int tile_rows, int tile_cols) {
  const int64_t m_tiles = (T + tile_rows - 1) / tile_rows, n_tiles = (N + tile_cols - 1) / tile_cols;
  const double x_bytes = 2.0 * T * K, w_bytes = 2.0 * K * N;
  int64_t R = (int64_t)(double(48 << 20) / (2.0 * tile_rows * K));
  int64_t C = (int64_t)(double(64 << 20) / (2.0 * tile_cols * K));
  R = R < 1 ? 1 : R > m_tiles ? m_tiles : R;
  C = C < 1 ? 1 : C > n_tiles ? n_tiles : C;
  Raster r;
  r.by_n = (x_bytes > double(128 << 20) && x_bytes >= 4.0 * w_bytes) ? 1 : 0;
  r.group = (int)(r.by_n ? C : R);
  if (const char* f = getenv("GEMM_EPI_RASTER")) {  // tuning override
    if (!strcmp(f, "m") || !strcmp(f, "n")) {
      r.by_n = f[0] == 'n';
      r.group = (int)(r.by_n ? C : R);
    }
  }
  if (const char* f = getenv("GEMM_EPI_GROUP_M")) {  // tuning override: the group size in tiles
    const int v = atoi(f);
    if (v >= 1) r.group = v;
  }
  const int64_t outer = r.by_n ? n_tiles : m_tiles;
  if (r.group > outer) r.group = (int)outer;
  return r;
}

// Clusters and CTAs of a kernel whose warps work alone (few_rows.cuh): `clusters` along
// the half rows of tiles, 2^split CTAs of each along the kt columns of tiles, at most
// `share` CTAs. What a launch takes goes by the half tiles of a warp (steps); a join over a
// cluster costs as much as `join` of them. No split where a warp would have more than two rows' sums.
struct FewChoice {
  int split = 0, clusters = 0;
  int64_t steps = 0;
};
inline FewChoice choose_few(const void* fn, int threads, uint32_t smem, int64_t N, int kt, int sms, int row_blocks, int join) {
  FewChoice best;
  const int halves = ceil_div(N, 16);
  int64_t cost = INT64_MAX;
  for (int split = 0; split <= 3 && 1 << split <= kt; ++split) {
    int clusters = (split == 0 ? sms : resident_clusters(fn, 1 << split, threads, smem, sms)) / row_blocks;
    if (clusters > halves) clusters = halves;
    if (clusters < 1) clusters = 1;  // (fewer SMs than blocks of rows: they take turns)
    const int64_t rows = ceil_div(halves, clusters);
    if (split > 0 && rows > ge::kFewWarps) break;
    const int64_t steps = (rows * ceil_div(kt, 1 << split) + ge::kFewWarps - 1) / ge::kFewWarps;
    if (steps + (split > 0 ? join : 0) >= cost) continue;
    cost = steps + (split > 0 ? join : 0);
    best.split = split;
    best.clusters = clusters;
    best.steps = steps;
  }
  return best;
}
inline ge::FewSplit few_split(const FewChoice& c, int64_t N, int kt) {
  const uint32_t halves = (uint32_t)ceil_div(N, 16), clusters = (uint32_t)c.clusters, ctas = 1u << c.split;
  return {c.split, halves / clusters, halves % clusters, (uint32_t)kt / ctas, (uint32_t)kt % ctas};
}

}  // namespace ge_host
