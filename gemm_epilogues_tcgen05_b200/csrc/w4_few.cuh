// w4_few.cuh -- few rows times a weight held in 4 bits (layout: w4_quant.cuh), each warp
// alone: Y[t][n] = epilog(sum_k X[t][k] s_g (q[n][k] - z_g)), and as a gated layer.
//
// With few rows the product is a pass over the codes. The kernel through tensor
// memory (w4_kernel.cuh) hands a block of columns on between four kinds of warps, 500 ns each time
// and 9 us before the first. Here every warp does all of it: it streams its own
// tiles of 32 features x 128 columns through its own ring in shared memory (cp.async,
// no barrier), unpacks them into the operands of mma.sync m16n8k16 (the
// features are its rows, the rows of X its eight columns), and scales a group's fp32
// sums. No weight is rounded anywhere.
//
// A word of the layout holds eight columns of one feature, and a lane takes the words of its
// features g, g + 8, ... and of the 8-column unit c (lane = 4 g + c): the order of the columns
// inside an MMA is free as long as X has the same one, and X's eight columns of a unit are
// 16 bytes of a row.
//
// Work split: clusters take runs of half rows of tiles (16 features), the CTAs of a
// cluster parts of the columns (only where a launch would have few CTAs: a cluster costs 2
// us), and a CTA's warps equal runs of its tiles, row after row. A row's sums meet once, at
// the end, in shared memory (distributed over the cluster), in a fixed order; no workspace.
// More rows of X than 16 (gridDim.y) are other CTAs', each 16 of them a pass over the codes.
//
// What bounds it is unpacking: seven instructions of half rate and four subtractions
// for eight bf16 weights (fp16: five and four); the MMAs take 2 cycles a quarter SM. N = 128000, K =
// 4096, T = 1, G = 128: 60.6 us, 4.4 TB/s, the ALU 61 % busy (with (w >> 4m & mask) | one
// left to the compiler, two instructions each, 73 us; shifts as multiplications, on the
// other pipe, 74). Small ones are bound by latency: K = 1024, N = 2048 3.5 us; K = 4096, N = 11008
// (22.5 MB, 3.6 us at the rate of a copy) 9.8, T = 8 10.8, T = 16 14.7, gated 14.5, 16.8, 21.2; shares of
// whole rows of tiles instead of half ones 10.7, 12.5, 16.6, gated 15.6, 17.9, 24.3. From
// 9 rows on X comes from L2 again and again, and the less shared memory the ring takes the
// more of it stays in L1: 3 places a warp 9.8 / 10.8 / 14.7 us for T = 1 / 8 / 16, 6 10.5 / 12.3 / 15.4.
#pragma once

#include "few_rows.cuh"
#include "w4_kernel.cuh"

namespace ge {

// NT: blocks of 8 rows of X; MATS: matrices; 128 / NG columns a group
template <int NT, int MATS, int NG, bool ZEROS>
struct W4Few {
  // a place of a warp's ring: codes, scales and zeros of a tile (of each matrix)
  static constexpr uint32_t TILE = kW4TileBytes + (ZEROS ? 96 : 64) * NG, PLACE = MATS * TILE;
  static constexpr int LD = kFewLd;
  static constexpr uint32_t SUMS = MATS * NT * 8 * LD * 4;      // of a warp and a row of tiles
  static constexpr int ROOM = (232448 / kFewWarps - 8 - SUMS) / PLACE;
  static constexpr int DEPTH = ROOM < 3 ? ROOM : 3;             // places of a warp's ring
  static constexpr uint32_t WARP = DEPTH * PLACE + SUMS;        // its last row's sums take the ring's place
  static constexpr uint32_t BYTES = kFewWarps * (WARP + 8);
  static_assert(DEPTH >= 2 && SUMS <= DEPTH * PLACE && PLACE % 16 == 0 && SUMS % 16 == 0, "ring");
  static_assert(BYTES <= 232448, "above the per-CTA limit");
};

template <int NT, bool GATED, int NG, bool ZEROS, bool BF16>
__global__ void __launch_bounds__(32 * kFewWarps, 1) w4_few_kernel(const W4MulParams p) {
  constexpr int MATS = GATED ? 2 : 1;
  using L = W4Few<NT, MATS, NG, ZEROS>;
  extern __shared__ __align__(16) uint8_t w4_smem[];
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3u;
  const uint32_t rank = blockIdx.x & ((1u << p.few.split) - 1u), cluster = blockIdx.x >> p.few.split;  // rank: along the columns
  const bool split = p.few.split > 0;
  // this cluster's half rows of tiles, this CTA's columns of them, this warp's tiles
  const uint32_t h0 = few_share(cluster, p.few.half_quot, p.few.half_rest), h1 = few_share(cluster + 1, p.few.half_quot, p.few.half_rest);
  const uint32_t kb0 = few_share(rank, p.few.kt_quot, p.few.kt_rest), nkb = few_share(rank + 1, p.few.kt_quot, p.few.kt_rest) - kb0;
  const FewRuns runs(h0, h1, nkb);
  const uint32_t row0 = runs.row0, u0 = runs.begin(warp), u1 = runs.begin(warp + 1);
  const int t0 = static_cast<int>(blockIdx.y) * (8 * NT), T = min(p.T - t0, 8 * NT);  // this CTA's rows of X
  uint8_t* ring = w4_smem + warp * L::WARP;
  // the rows of tiles whose sums a warp keeps: the first, the last
  int* kept = reinterpret_cast<int*>(w4_smem + kFewWarps * L::WARP);
  if (lane < 2) kept[2 * warp + lane] = -1;
  __syncwarp();
  wait_for_inputs();

  // ---- copies: unit u is tile (row0 + u / nkb, kb0 + u % nkb)
  const uint64_t policy = l2_policy_evict_first();
  uint32_t row = u0 / nkb, kb = u0 - row * nkb;  // of the next unit's work
  uint32_t in_kb = kb, in = u0, in_place = smem_u32(ring) + lane * 16;  // of the next unit's copies
  const uint32_t ring_end = in_place + L::DEPTH * L::PLACE;
  // 16 bytes a lane of each kind: codes, then the first 4 NG lanes scales, the next 2 NG zeros
  const int64_t tile0 = static_cast<int64_t>(row0 + row) * p.kt + kb0 + kb, matrix = static_cast<int64_t>(p.rt) * p.kt;
  const uint8_t* q = p.q + tile0 * kW4TileBytes + lane * 16;
  uint32_t in_row = row;
  const bool side_scales = lane < 4 * NG, side_in = lane < (ZEROS ? 6 : 4) * NG;
  const uint32_t side_bytes = side_scales ? 64 * NG : 32 * NG;
  const uint8_t* side = side_scales ? reinterpret_cast<const uint8_t*>(p.scales) + tile0 * (64 * NG) + lane * 16
                                    : p.zeros + tile0 * (32 * NG) + (lane - 4 * NG) * 16;
  const auto fetch = [&]() {
    if (in < u1) {
      // (features 0 .. 15 are the lower lanes', and the half that another CTA takes is left out)
      const bool wanted = 2 * (row0 + in_row) + (lane >> 4) - h0 < h1 - h0;
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (wanted) w4_copy_16(in_place + m * L::TILE + 512 * b, q + m * matrix * kW4TileBytes + 512 * b, policy);
        if (side_in) w4_copy_16(in_place + m * L::TILE + kW4TileBytes, side + m * matrix * side_bytes, policy);
      }
      in_place = in_place + L::PLACE == ring_end ? ring_end - L::DEPTH * L::PLACE : in_place + L::PLACE;
      q += kW4TileBytes;
      side += side_bytes;
      ++in;
      if (++in_kb == nkb) {
        in_kb = 0;
        ++in_row;
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

  const uint4* X = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.X) + (static_cast<int64_t>(t0) + g) * p.K + c * 8);
  const int64_t x_step = p.K;  // 8 rows, in units of 8 columns
  // a tile's products, of its halves from .. to - 1
  const auto multiply = [&](const uint8_t* place, const uint4 (&x)[4][NT], auto from, auto to) {
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int h = decltype(from)::value; h < decltype(to)::value; ++h) {
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
              few_mma<BF16>(part[t], b == k * PER, r[0], r[4], r[1], r[5], x[b][t].x, x[b][t].y);
              few_mma<BF16>(part[t], false, r[2], r[6], r[3], r[7], x[b][t].z, x[b][t].w);
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
  };
  const uint8_t* place = ring;
  uint32_t seg_kb = kb;
  for (uint32_t u = u0; u < u1; ++u) {
    uint4 x[4][NT];
    {
      const uint4* xk = X + (kb0 + kb) * 16;
      const int left = p.K - static_cast<int>(kb0 + kb) * 128;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int blocks = t * 8 + static_cast<int>(g) < T ? left : 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) x[b][t] = b * 32 < blocks ? xk[t * x_step + b * 4] : make_uint4(0, 0, 0, 0);
      }
    }
    cp_async_wait<L::DEPTH - 1>();
    __syncwarp();
    const uint32_t half = 2 * (row0 + row);
    if (half >= h0 && half + 1 < h1)
      multiply(place, x, FewHalf<0>(), FewHalf<2>());
    else if (half >= h0)
      multiply(place, x, FewHalf<0>(), FewHalf<1>());
    else
      multiply(place, x, FewHalf<1>(), FewHalf<2>());
    __syncwarp();  // the place has been read
    fetch();
    place = place + L::PLACE == ring + L::DEPTH * L::PLACE ? ring : place + L::PLACE;
    // the end of a row of tiles: a whole row that needs no other warp is finished, the
    // first row's and the last row's sums are kept
    if (++kb < nkb && u + 1 < u1) continue;
    if (!split && seg_kb == 0 && kb == nkb) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const int n = static_cast<int>((row0 + row) * 32 + 16 * h + g + 4 * e);
          if (n >= p.N || 2 * (row0 + row) + h - h0 >= h1 - h0) continue;
          const float bias_a = bias_of(n), bias_b = GATED ? bias_of(p.N + n) : 0.f;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (t * 8 + static_cast<int>(2 * c) + i < T)
                w4_output<GATED, BF16>(p, acc[0][t][h][e + i], acc[MATS - 1][t][h][e + i], t0 + t * 8 + 2 * c + i, n, bias_a, bias_b);
        }
    } else {
      const bool last = u + 1 == u1;
      stash(last ? ring : ring + L::DEPTH * L::PLACE);
      if (lane == 0) kept[2 * warp + last] = static_cast<int>(row);
    }
    clear();
    kb = seg_kb = 0;
    ++row;
  }
  cp_async_wait<0>();
  few_join<NT, MATS, L::WARP, L::DEPTH * L::PLACE>(
      w4_smem, p.few.split, rank, T, [&](uint32_t r, uint32_t t, float a, float b) {
        const uint32_t half = 2 * (row0 + r) + (lane >> 4);
        const int n = static_cast<int>((row0 + r) * 32 + lane);
        if (half >= h0 && half < h1 && n < p.N)
          w4_output<GATED, BF16>(p, a, b, t0 + static_cast<int>(t), n, bias_of(n), GATED ? bias_of(p.N + n) : 0.f);
      });
}

}  // namespace ge
