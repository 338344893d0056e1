// w4_few.cuh -- at most 16 rows times a weight held in 4 bits (layout: w4_quant.cuh).
//
// With so few rows the product is a pass over the codes, and what costs is the way to
// them: the kernel of more rows (w4_kernel.cuh) hands a block on between four kinds of
// warps. Here every warp does all of it alone: it streams its own tiles of 32 features
// x 128 columns through its own ring in shared memory (bulk copies, one barrier a
// place), so that an SM has up to 200 KB under way from the first cycle, unpacks them into the
// operands of mma.sync m16n8k16 (the features are its rows, the rows of X its eight
// columns), and scales a group's sums in fp32. Tensor memory has no part in it:
// 27 cycles a quarter SM for each of these MMAs are less than the stages cost there.
//
// A word of the layout holds eight columns of one feature, and a lane takes the words of its
// features g, g + 8, ... and of the 8-column unit c (lane = 4 g + c): the order of the columns
// inside an MMA is free as long as X has the same one, and X's eight columns of a unit are
// 16 bytes of a row.
//
// Work split: clusters take runs of 32-feature rows of tiles, the CTAs of a cluster
// parts of the columns, and a CTA's warps equal runs of its tiles, row after row. A
// row's sums meet once, at the end, in shared memory (distributed over the cluster), in
// a fixed order; no workspace.
#pragma once

#include "w4_kernel.cuh"

namespace ge {

constexpr int kW4FewWarps = 16;

// NT: blocks of 8 rows of X; MATS: matrices; 128 / NG columns a group
template <int NT, int MATS, int NG, bool ZEROS>
struct W4Few {
  // a place of a warp's ring: codes, scales and zeros of a tile (of each matrix)
  static constexpr uint32_t TILE = kW4TileBytes + (ZEROS ? 96 : 64) * NG, PLACE = MATS * TILE;
  static constexpr int LD = 36;                                 // floats between a sum's rows: no two lanes in a bank
  static constexpr uint32_t SUMS = MATS * NT * 8 * LD * 4;      // of a warp and a row of tiles
  static constexpr int ROOM = (232448 / kW4FewWarps - SUMS) / PLACE;
  static constexpr int DEPTH = ROOM < 6 ? ROOM : 6;             // places of a warp's ring
  static constexpr uint32_t WARP = DEPTH * PLACE + SUMS;        // its last row's sums take the ring's place
  static constexpr uint32_t BYTES = kW4FewWarps * WARP;
  static_assert(DEPTH >= 2 && SUMS <= DEPTH * PLACE && PLACE % 16 == 0 && SUMS % 16 == 0, "ring");
  static_assert(BYTES <= 232448, "above the per-CTA limit");
};

template <bool BF16>
__device__ __forceinline__ void w4_mma(float (&d)[4], bool zero, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  const float c0 = zero ? 0.f : d[0], c1 = zero ? 0.f : d[1], c2 = zero ? 0.f : d[2], c3 = zero ? 0.f : d[3];
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// first of `total` units of part `i` of `parts` (the plan keeps the products below 2^31)
__device__ __forceinline__ uint32_t w4_share(uint32_t total, uint32_t i, uint32_t parts) { return total * i / parts; }

template <int NT, bool GATED, int NG, bool ZEROS, bool BF16>
__global__ void __launch_bounds__(32 * kW4FewWarps, 1) w4_few_kernel(const W4MulParams p) {
  constexpr int MATS = GATED ? 2 : 1, W = kW4FewWarps;
  using L = W4Few<NT, MATS, NG, ZEROS>;
  extern __shared__ __align__(16) uint8_t w4_smem[];
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3u;
  const uint32_t split = static_cast<uint32_t>(p.split), rank = blockIdx.x % split;  // CTAs of a cluster, along the columns
  const uint32_t cluster = blockIdx.x / split, clusters = gridDim.x / split;
  // this cluster's rows of tiles, this CTA's columns of them, this warp's tiles
  const uint32_t row0 = w4_share(p.rt, cluster, clusters), rows = w4_share(p.rt, cluster + 1, clusters) - row0;
  const uint32_t kb0 = w4_share(p.kt, rank, split), nkb = w4_share(p.kt, rank + 1, split) - kb0;
  const uint32_t units = rows * nkb, parts = min(units, static_cast<uint32_t>(W));
  const uint32_t u0 = warp < parts ? w4_share(units, warp, parts) : units, u1 = warp < parts ? w4_share(units, warp + 1, parts) : units;
  uint8_t* ring = w4_smem + warp * L::WARP;
  wait_for_inputs();

  // ---- copies: unit u is tile (row0 + u / nkb, kb0 + u % nkb)
  const uint64_t policy = l2_policy_evict_first();
  uint32_t row = u0 / nkb, kb = u0 - row * nkb;  // of the next unit's work
  uint32_t in_kb = kb, in = u0, in_place = smem_u32(ring) + lane * 16;  // of the next unit's copies
  const uint32_t ring_end = in_place + L::DEPTH * L::PLACE;
  // 16 bytes a lane of each kind: codes, then the first 4 NG lanes scales, the next 2 NG zeros
  const int64_t tile0 = static_cast<int64_t>(row0 + row) * p.kt + kb0 + kb, matrix = static_cast<int64_t>(p.rt) * p.kt;
  const uint8_t* q = p.q + tile0 * kW4TileBytes + lane * 16;
  const bool side_scales = lane < 4 * NG, side_in = lane < (ZEROS ? 6 : 4) * NG;
  const uint32_t side_bytes = side_scales ? 64 * NG : 32 * NG;
  const uint8_t* side = side_scales ? reinterpret_cast<const uint8_t*>(p.scales) + tile0 * (64 * NG) + lane * 16
                                    : p.zeros + tile0 * (32 * NG) + (lane - 4 * NG) * 16;
  const auto fetch = [&]() {
    if (in < u1) {
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          w4_copy_16(in_place + m * L::TILE + 512 * b, q + m * matrix * kW4TileBytes + 512 * b, policy);
        if (side_in) w4_copy_16(in_place + m * L::TILE + kW4TileBytes, side + m * matrix * side_bytes, policy);
      }
      in_place = in_place + L::PLACE == ring_end ? ring_end - L::DEPTH * L::PLACE : in_place + L::PLACE;
      q += kW4TileBytes;
      side += side_bytes;
      ++in;
      if (++in_kb == nkb) {
        in_kb = 0;
        q += static_cast<int64_t>(p.kt - nkb) * kW4TileBytes;
        side += static_cast<int64_t>(p.kt - nkb) * side_bytes;
      }
    }
    cp_async_commit();
  };
  for (int d = 0; d < L::DEPTH; ++d) fetch();

  float acc[MATS][NT][2][4];
  const auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MATS * NT * 8; ++i) (&acc[0][0][0][0])[i] = 0.f;
  };
  clear();
  // a row's sums of this warp: [matrix][row of X][feature]
  const auto stash = [&](uint8_t* to) {
    float* at = reinterpret_cast<float*>(to) + 2 * c * L::LD + g;
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) at[((m * NT + t) * 8 + (e & 1)) * L::LD + 16 * h + 8 * (e >> 1)] = acc[m][t][h][e];
  };
  const auto bias_of = [&](uint32_t n) { return p.bias ? load_bias<BF16>(p.bias, p.bias_f32, n) : 0.f; };

  const uint4* X = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.X) + static_cast<int64_t>(g) * p.K + c * 8);
  const int64_t x_step = p.K;  // 8 rows, in units of 8 columns
  const uint8_t* place = ring;
  uint32_t seg_kb = kb;
  for (uint32_t u = u0; u < u1; ++u) {
    uint4 x[4][NT];
    {
      const uint4* xk = X + (kb0 + kb) * 16;
      const int left = p.K - static_cast<int>(kb0 + kb) * 128;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int blocks = t * 8 + static_cast<int>(g) < p.T ? left : 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) x[b][t] = b * 32 < blocks ? __ldg(xk + t * x_step + b * 4) : make_uint4(0, 0, 0, 0);
      }
    }
    cp_async_wait<L::DEPTH - 1>();
    __syncwarp();
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* tile = place + m * L::TILE;
        const uint32_t f = 16 * h + g;
        float part[NT][4];
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          constexpr int PER = 4 / NG;  // 32-column blocks of a group
          const uint8_t* z = tile + kW4TileBytes + 64 * NG + 32 * k + f;
          const W4Unpack<BF16> lo(ZEROS ? z[0] : 8u), hi(ZEROS ? z[8] : 8u);
#pragma unroll
          for (int b = k * PER; b < (k + 1) * PER; ++b) {
            const uint32_t* word = reinterpret_cast<const uint32_t*>(tile + 512 * b + 16 * f + 4 * c);
            uint32_t r[8];
            lo(word[0], r, 0);
            hi(word[32], r, 4);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              w4_mma<BF16>(part[t], b == k * PER, r[0], r[4], r[1], r[5], x[b][t].x, x[b][t].y);
              w4_mma<BF16>(part[t], false, r[2], r[6], r[3], r[7], x[b][t].z, x[b][t].w);
            }
          }
          const uint16_t* sc = reinterpret_cast<const uint16_t*>(tile + kW4TileBytes + 64 * k + 2 * f);
          const float s0 = w4_float<BF16>(sc[0]), s1 = w4_float<BF16>(sc[8]);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][t][h][e] = fmaf(e < 2 ? s0 : s1, part[t][e], acc[m][t][h][e]);
        }
      }
    __syncwarp();  // the place has been read
    fetch();
    place = place + L::PLACE == ring + L::DEPTH * L::PLACE ? ring : place + L::PLACE;
    // the end of a row of tiles: a whole row that needs no other warp is finished, the
    // first row's and the last row's sums are kept
    if (++kb < nkb && u + 1 < u1) continue;
    if (split == 1 && seg_kb == 0 && kb == nkb) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const int n = static_cast<int>((row0 + row) * 32 + 16 * h + g + 4 * e);
          if (n >= p.N) continue;
          const float bias_a = bias_of(n), bias_b = GATED ? bias_of(p.N + n) : 0.f;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (t * 8 + static_cast<int>(2 * c) + i < p.T)
                w4_output<GATED, BF16>(p, acc[0][t][h][e + i], acc[MATS - 1][t][h][e + i], t * 8 + 2 * c + i, n, bias_a, bias_b);
        }
    } else {
      stash(u + 1 == u1 ? ring : ring + L::DEPTH * L::PLACE);
    }
    clear();
    kb = seg_kb = 0;
    ++row;
  }
  cp_async_wait<0>();
  __syncwarp();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();

  // ---- the rows that several warps share: outputs (row, t, feature), the CTAs of a
  // cluster in turn
  const uint32_t outs = rows * static_cast<uint32_t>(p.T) * 32;
  for (uint32_t o = threadIdx.x + rank * (32 * W); o < outs; o += 32 * W * split) {
    const uint32_t f = o & 31u, rt = o >> 5, r = rt / static_cast<uint32_t>(p.T), t = rt - r * static_cast<uint32_t>(p.T);
    float a = 0.f, b = 0.f;
    bool whole = false;
    for (uint32_t s = 0; s < split; ++s) {
      const uint32_t n = w4_share(p.kt, s + 1, split) - w4_share(p.kt, s, split), total = rows * n;
      const uint32_t among = min(total, static_cast<uint32_t>(W));
      const uint32_t base = split > 1 ? mapa_shared(smem_u32(w4_smem), s) : smem_u32(w4_smem);
      uint32_t w = skinny_owner32(r * n, among, total);
      const uint32_t last = skinny_owner32((r + 1) * n - 1, among, total);
      whole = split == 1 && w == last;
      if (whole) break;
      for (; w <= last; ++w) {
        const bool ends = w4_share(total, w + 1, among) <= (r + 1) * n;  // it is this warp's last row
        const uint32_t at = base + w * L::WARP + (ends ? 0 : L::DEPTH * L::PLACE) + (t * L::LD + f) * 4;
        a += ld_cluster_f32(at);
        if constexpr (GATED) b += ld_cluster_f32(at + NT * 8 * L::LD * 4);
      }
    }
    const int n = static_cast<int>((row0 + r) * 32 + f);
    if (whole || n >= p.N) continue;
    w4_output<GATED, BF16>(p, a, b, t, n, bias_of(n), GATED ? bias_of(p.N + n) : 0.f);
  }
  __syncwarp();
  if (split > 1) cluster_sync();  // (sums that another CTA reads)
}

}  // namespace ge
