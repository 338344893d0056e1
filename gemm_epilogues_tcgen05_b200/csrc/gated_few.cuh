// gated_few.cuh -- gated layer of at most 16 rows, each warp alone: Z = X W + b, H = act(Zg) Zu.
//
// As w4_few.cuh, of a 16-bit weight: every warp streams units of 32 features x 32
// columns of both halves of the weight (4 KB) through its own ring in shared memory and
// multiplies them with mma.sync m16n8k16, the features as its rows; no tensor memory, no
// barriers, sums that meet once in shared memory. The order of the columns inside an MMA is
// free as long as X has the same one: lane 4 g + c holds columns 8 c .. 8 c + 7 of a unit, 16
// bytes of a row of X. N x K weights: a lane copies and reads its own 16-byte pieces
// (features g, g + 8, ...). K x N weights: rows of 64 bytes, piece q of row k at q ^ (k / 8), so
// that the transposing ldmatrix, whose eight rows are two columns each of four lanes, is
// free of bank conflicts.
//
// For small weights, where a launch is mostly latency: K = 1024, N = 2048 (8.4 MB, 1.3 us at
// the rate of a copy), T = 1 4.6 us N x K, 5.1 K x N, where the few-row kernel's barriers,
// tensor memory and join through a workspace take 6.6. Large ones stream better by TMA: K =
// 4096, N = 11008 38 us here (pieces of 64 bytes; K x N 54), 31.8 there; the plan has the rule.
#pragma once

#include "activation.cuh"
#include "few_rows.cuh"
#include "tile_kernel.cuh"

namespace ge {

struct GatedFewParams {
  int32_t T, N, K;
  int32_t act;
  int32_t bias_f32, out_f32;
  FewSplit few;  // of units of 32 columns
  const void* X;
  const void* W;
  const void* bias;
  void* out;
  void* aux_out;  // or null
};

template <int NT>
struct GatedFew {
  static constexpr uint32_t PLACE = 4096;                   // [matrix] 2048 bytes
  static constexpr uint32_t SUMS = 2 * NT * 8 * kFewLd * 4; // of a warp and a row of units
  static constexpr int DEPTH = 2;
  static constexpr uint32_t WARP = DEPTH * PLACE + SUMS;
  static constexpr uint32_t BYTES = kFewWarps * (WARP + 8);
  static_assert(SUMS <= DEPTH * PLACE && BYTES <= 232448, "shared memory");
};

// 16 bytes, or zeros
__device__ __forceinline__ void few_copy_16(uint32_t saddr, const void* src, bool in, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(saddr), "l"(src), "r"(in ? 16 : 0),
               "l"(policy)
               : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t saddr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}

template <bool BF16>
__device__ __forceinline__ void gated_few_output(const GatedFewParams& p, float g, float u, int t, int n, float bias_g,
                                                 float bias_u) {
  g += bias_g;
  u += bias_u;
  const uint32_t both = pack2<BF16>(g, u);
  if (p.aux_out) {
    uint16_t* z = reinterpret_cast<uint16_t*>(p.aux_out) + static_cast<int64_t>(t) * 2 * p.N + n;
    z[0] = static_cast<uint16_t>(both & 0xffffu);
    z[p.N] = static_cast<uint16_t>(both >> 16);
  }
  float z[2] = {g, g}, v[2], none[2];
  act_values<2, false>(p.act, z, v, none);
  const int64_t o = static_cast<int64_t>(t) * p.N + n;
  if (p.out_f32)
    reinterpret_cast<float*>(p.out)[o] = v[0] * u;
  else
    reinterpret_cast<uint16_t*>(p.out)[o] = static_cast<uint16_t>(pack2<BF16>(v[0] * u, 0.f) & 0xffffu);
}

template <int NT, bool NK, bool BF16>
__global__ void __launch_bounds__(32 * kFewWarps, 1) gated_few_kernel(const GatedFewParams p) {
  using L = GatedFew<NT>;
  extern __shared__ __align__(16) uint8_t few_smem[];
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3u;
  const uint32_t rank = blockIdx.x & ((1u << p.few.split) - 1u), cluster = blockIdx.x >> p.few.split;
  const bool split = p.few.split > 0;
  const uint32_t h0 = few_share(cluster, p.few.half_quot, p.few.half_rest), h1 = few_share(cluster + 1, p.few.half_quot, p.few.half_rest);
  const uint32_t kb0 = few_share(rank, p.few.kt_quot, p.few.kt_rest), nkb = few_share(rank + 1, p.few.kt_quot, p.few.kt_rest) - kb0;
  const FewRuns runs(h0, h1, nkb);
  const uint32_t row0 = runs.row0, u0 = runs.begin(warp), u1 = runs.begin(warp + 1);
  uint8_t* ring = few_smem + warp * L::WARP;
  int* kept = reinterpret_cast<int*>(few_smem + kFewWarps * L::WARP);
  if (lane < 2) kept[2 * warp + lane] = -1;
  __syncwarp();
  wait_for_inputs();

  // ---- copies: unit u is (row0 + u / nkb, kb0 + u % nkb)
  const uint64_t policy = l2_policy_evict_first();
  uint32_t row = u0 / nkb, kb = u0 - row * nkb;          // of the next unit's work
  uint32_t in_row = row, in_kb = kb, in = u0, in_place = 0;  // of the next unit's copies
  const uint32_t ring_at = smem_u32(ring);
  const uint16_t* W = reinterpret_cast<const uint16_t*>(p.W);
  const auto fetch = [&]() {
    if (in < u1) {
      const uint32_t at = ring_at + in_place * L::PLACE;
      const int n0 = static_cast<int>(row0 + in_row) * 32, k0 = static_cast<int>(kb0 + in_kb) * 32;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (the half that another CTA takes is not read, nor copied)
          if constexpr (NK) {
            const int n = n0 + 8 * i + static_cast<int>(g), k = k0 + 8 * static_cast<int>(c);
            const uint32_t half = static_cast<uint32_t>(n0 / 16 + i / 2);
            const bool ok = half - h0 < h1 - h0 && n < p.N && k < p.K;
            few_copy_16(at + m * 2048 + i * 512 + lane * 16, W + (ok ? (static_cast<int64_t>(m) * p.N + n) * p.K + k : 0), ok, policy);
          } else {
            const int kk = 8 * i + static_cast<int>(g), k = k0 + kk, n = n0 + 8 * static_cast<int>(c);
            const uint32_t half = static_cast<uint32_t>(n0 / 16) + c / 2;
            const bool ok = half - h0 < h1 - h0 && n < p.N && k < p.K;
            few_copy_16(at + m * 2048 + kk * 64 + ((c ^ i) * 16), W + (ok ? static_cast<int64_t>(k) * 2 * p.N + static_cast<int64_t>(m) * p.N + n : 0), ok, policy);
          }
        }
      in_place = in_place + 1 == L::DEPTH ? 0 : in_place + 1;
      ++in;
      if (++in_kb == nkb) {
        in_kb = 0;
        ++in_row;
      }
    }
    cp_async_commit();
  };
  for (int d = 0; d < L::DEPTH; ++d) fetch();

  float acc[2][NT][2][4];
  const auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 2 * NT * 8; ++i) (&acc[0][0][0][0])[i] = 0.f;
  };
  clear();
  const auto stash = [&](uint8_t* to) {
    float* at = reinterpret_cast<float*>(to) + 2 * c * kFewLd + g;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) at[((m * NT + t) * 8 + (e & 1)) * kFewLd + 16 * h + 8 * (e >> 1)] = acc[m][t][h][e];
  };
  const auto bias_of = [&](int64_t n) { return p.bias ? load_bias<BF16>(p.bias, p.bias_f32, n) : 0.f; };
  const auto load_x = [&](uint4 (&x)[NT], uint32_t block) {
    const int k = static_cast<int>(kb0 + block) * 32 + 8 * static_cast<int>(c);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      x[t] = t * 8 + static_cast<int>(g) < p.T && k < p.K
                 ? *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.X) +
                                                   static_cast<int64_t>(t * 8 + static_cast<int>(g)) * p.K + k)
                 : make_uint4(0, 0, 0, 0);
  };
  // rows of ldmatrix: column 8 (r / 2) + r % 2 of matrix lane / 8, row r = lane % 8
  const uint32_t mi = lane >> 3, kk0 = 8 * ((lane & 7u) >> 1) + (lane & 1u) + 2 * (mi >> 1);
  uint32_t place = 0, seg_kb = kb;
  uint4 x[NT];
  if (u0 < u1) load_x(x, kb);
  for (uint32_t u = u0; u < u1; ++u) {
    uint4 next[NT];
    const uint32_t next_kb = kb + 1 == nkb ? 0 : kb + 1;
    if (u + 1 < u1) load_x(next, next_kb);
    cp_async_wait<L::DEPTH - 1>();
    if constexpr (!NK) __syncwarp();
    const uint32_t at = ring_at + place * L::PLACE, half = 2 * (row0 + row);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (half + h - h0 >= h1 - h0) continue;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t a0[4], a1[4];
        if constexpr (NK) {
          const uint4 lo = ld_shared_v4(at + m * 2048 + (2 * h) * 512 + lane * 16);
          const uint4 hi = ld_shared_v4(at + m * 2048 + (2 * h + 1) * 512 + lane * 16);
          a0[0] = lo.x, a0[1] = hi.x, a0[2] = lo.y, a0[3] = hi.y;
          a1[0] = lo.z, a1[1] = hi.z, a1[2] = lo.w, a1[3] = hi.w;
        } else {
          const uint32_t piece = ((2 * h + (mi & 1u)) ^ ((lane & 7u) >> 1)) * 16;
          ldmatrix_x4_trans(a0, at + m * 2048 + kk0 * 64 + piece);
          ldmatrix_x4_trans(a1, at + m * 2048 + (kk0 + 4) * 64 + piece);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          few_mma<BF16>(acc[m][t][h], false, a0[0], a0[1], a0[2], a0[3], x[t].x, x[t].y);
          few_mma<BF16>(acc[m][t][h], false, a1[0], a1[1], a1[2], a1[3], x[t].z, x[t].w);
        }
      }
    }
    if constexpr (!NK) __syncwarp();  // the place has been read
    fetch();
    place = place + 1 == L::DEPTH ? 0 : place + 1;
#pragma unroll
    for (int t = 0; t < NT; ++t) x[t] = next[t];
    if (++kb < nkb && u + 1 < u1) continue;
    if (!split && seg_kb == 0 && kb == nkb) {  // a whole row: no other warp has a part
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const int n = static_cast<int>((row0 + row) * 32 + 16 * h + g + 4 * e);
          if (n >= p.N || half + h - h0 >= h1 - h0) continue;
          const float bias_g = bias_of(n), bias_u = bias_of(static_cast<int64_t>(p.N) + n);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (t * 8 + static_cast<int>(2 * c) + i < p.T)
                gated_few_output<BF16>(p, acc[0][t][h][e + i], acc[1][t][h][e + i], t * 8 + 2 * c + i, n, bias_g, bias_u);
        }
    } else {
      const bool last = u + 1 == u1;
      if (last) {
        cp_async_wait<0>();
        __syncwarp();  // the ring has been read
      }
      stash(last ? ring : ring + L::DEPTH * L::PLACE);
      if (lane == 0) kept[2 * warp + last] = static_cast<int>(row);
    }
    clear();
    kb = seg_kb = 0;
    ++row;
  }
  cp_async_wait<0>();
  few_join<NT, 2, L::WARP, L::DEPTH * L::PLACE>(few_smem, p.few.split, rank, p.T, [&](uint32_t r, uint32_t t, float a, float b) {
    const uint32_t half = 2 * (row0 + r) + (lane >> 4);
    const int n = static_cast<int>((row0 + r) * 32 + lane);
    if (half >= h0 && half < h1 && n < p.N)
      gated_few_output<BF16>(p, a, b, static_cast<int>(t), n, bias_of(n), bias_of(static_cast<int64_t>(p.N) + n));
  });
}

}  // namespace ge
