// gated_epilogue.cuh -- epilogues of a gated layer for the tile kernels (one
// CTA and CTA pairs), and of its backward.
//
//   GATED   Z = X W + b, W of 2N columns: N of the gate, then N of the up
//           projection. H[t][n] = act(Z[t][n]) Z[t][N + n]; Z may be stored
//           (16-bit, T x 2N) for the backward.
//   DGATED  dH = dY W2; with G | U = Z as stored: dG = dH U act'(G), dU = dH
//           act(G), dZ = [dG | dU] (T x 2N); optionally the column sums of dZ
//           before its rounding (the bias gradient, 2N).
//
// A gated tile's accumulator holds the gate's pre-activations of some features
// in one half of its columns and the up projection's of the same features in
// the other (on a CTA pair, each CTA loads the weight of one half), so that a
// thread finds both in its own row of tensor memory and H never needs a second
// kernel: the layer's 2N pre-activations go out once, for the backward, or not
// at all. Z and dZ go out as matrices of N columns, two a row (3-D tensor
// maps), so that a block of 32 columns is cut at N in each half.
//
// Beside the products, DGATED reads and writes 2 x 4TN bytes: at T = K = 4096,
// N = 11008 361 of its 484 MB, 74 us at the copy rate under 226 us of MMA.
#pragma once

#include "activation.cuh"
#include "ptx.cuh"

namespace ge {

// The tile's bias values (fp32; zeros without a bias): the gate's at bs[0 ..],
// the up projection's at bs[BN / 2 ..].
template <int BN, bool BF16, int NT>
__device__ __forceinline__ void gated_stage_bias(const TileParams& p, int n0, float* bs, uint32_t et, int ncols) {
  for (int c = et; c < 2 * ncols; c += NT) {
    const int half = c >= ncols ? 1 : 0, cc = c - half * ncols, n = n0 + cc;
    bs[half * (BN / 2) + cc] =
        p.bias && n < p.N ? load_bias<BF16>(p.bias, p.bias_f32, static_cast<int64_t>(half) * p.N + n) : 0.f;
  }
}

// A warp's 32 x 32 block (row = lane) through one of its staging buffers, as in
// store_block16, to column x and row y of a 2-D map or of matrix `half` of a
// 3-D one; fp32 outputs as two blocks of 16 columns, cut at p.N.
template <bool BF16, int NB, bool THREE_D>
__device__ __forceinline__ void gated_store(const float (&v)[32], const CUtensorMap* map, uint8_t* stg, uint32_t& scount,
                                            int x, int half, int y, bool f32, int N) {
  const uint32_t lane = lane_id();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 1 && (!f32 || x + 16 >= N)) break;  // warp-uniform
    uint8_t* buf = stg + scount * 2048;
    if (lane == 0) bulk_wait_group_read<NB - 1>();
    __syncwarp();
    const uint32_t rbase = smem_u32(buf) + lane * 64;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 w;
      if (f32)
        w = make_uint4(__float_as_uint(v[16 * h + 4 * q]), __float_as_uint(v[16 * h + 4 * q + 1]),
                       __float_as_uint(v[16 * h + 4 * q + 2]), __float_as_uint(v[16 * h + 4 * q + 3]));
      else
        w = make_uint4(pack2<BF16>(v[8 * q], v[8 * q + 1]), pack2<BF16>(v[8 * q + 2], v[8 * q + 3]),
                       pack2<BF16>(v[8 * q + 4], v[8 * q + 5]), pack2<BF16>(v[8 * q + 6], v[8 * q + 7]));
      st_shared_v4(rbase + ((q ^ ((lane >> 1) & 3u)) * 16), w);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if constexpr (THREE_D)
        tma_store_3d(map, buf, x + 16 * h, half, y);
      else
        tma_store_2d(map, buf, x + 16 * h, y);
      bulk_commit_group();
    }
    scount = scount + 1 == NB ? 0 : scount + 1;
  }
}

// Forward: this warp's 32 rows, output columns n0 .. n0 + ncols - 1, whose gate
// is at TMEM address tgate and whose up projection at tup.
template <bool BF16, int NB>
__device__ __forceinline__ void gated_rows(const TileParams& p, uint32_t tgate, uint32_t tup, int n0, int ncols,
                                           const float* bgate, const float* bup, const CUtensorMap* tmY,
                                           const CUtensorMap* tmAux, uint8_t* stg, uint32_t& scount, int wrow0) {
#pragma unroll 1
  for (int c = 0; c < ncols; c += 32) {
    const int nc0 = n0 + c;
    if (nc0 >= p.N) break;  // warp-uniform
    uint32_t rg[32], ru[32];
    tmem_ld_32x32b_x32(tgate + c, rg);
    tmem_ld_32x32b_x32(tup + c, ru);
    tmem_wait_ld();
    float g[32], u[32], none[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      g[j] = __uint_as_float(rg[j]) + bgate[c + j];
      u[j] = __uint_as_float(ru[j]) + bup[c + j];
    }
    if (p.aux_out) {
      gated_store<BF16, NB, true>(g, tmAux, stg, scount, nc0, 0, wrow0, false, p.N);
      gated_store<BF16, NB, true>(u, tmAux, stg, scount, nc0, 1, wrow0, false, p.N);
    }
    act_values<32, false>(p.act, g, g, none);
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] *= u[j];
    gated_store<BF16, NB, false>(g, tmY, stg, scount, nc0, 0, wrow0, p.out_f32 != 0, p.N);
  }
}

// Backward: 32 columns of G and of U of one row, 16-bit.
struct DGatedInput {
  uint4 g[4], u[4];
};

__device__ __forceinline__ DGatedInput dgated_load(const TileParams& p, int row, int nc0) {
  DGatedInput r;
  const uint16_t* z = reinterpret_cast<const uint16_t*>(p.aux_in) + static_cast<int64_t>(row) * 2 * p.N + nc0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const bool in = row < p.T && nc0 + 8 * q < p.N;  // N is a multiple of 8
    r.g[q] = in ? __ldg(reinterpret_cast<const uint4*>(z + 8 * q)) : make_uint4(0, 0, 0, 0);
    r.u[q] = in ? __ldg(reinterpret_cast<const uint4*>(z + p.N + 8 * q)) : make_uint4(0, 0, 0, 0);
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ void unpack_2x(uint32_t w, float& lo, float& hi) {
  if constexpr (BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    lo = __low2float(h);
    hi = __high2float(h);
  }
}

// This warp's 32 rows (row = this lane's), columns n0 .. n0 + ncols - 1, of which `in`
// holds the first 32 of G and U: each next 32 are loaded while the last are
// worked on. colp (fp32, this lane quarter's): the column sums, dG's and, `gap` later, dU's.
template <bool BF16, int NB>
__device__ __forceinline__ void dgated_rows(const TileParams& p, uint32_t tbase, int row, int n0, int ncols,
                                            DGatedInput in, float* colp, int gap, const CUtensorMap* tmY, uint8_t* stg,
                                            uint32_t& scount, int wrow0) {
  const uint32_t lane = lane_id();
#pragma unroll 1
  for (int c = 0; c < ncols; c += 32) {
    const int nc0 = n0 + c;
    if (nc0 >= p.N) break;  // warp-uniform
    uint32_t r[32];
    tmem_ld_32x32b_x32(tbase + c, r);
    tmem_wait_ld();
    float dg[32], du[32];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t wg[4] = {in.g[q].x, in.g[q].y, in.g[q].z, in.g[q].w};
      const uint32_t wu[4] = {in.u[q].x, in.u[q].y, in.u[q].z, in.u[q].w};
      float g[8], a[8], d[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack_2x<BF16>(wg[j], g[2 * j], g[2 * j + 1]);
      act_values<8, true>(p.act, g, a, d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float u0, u1;
        unpack_2x<BF16>(wu[j], u0, u1);
        const float h0 = __uint_as_float(r[8 * q + 2 * j]), h1 = __uint_as_float(r[8 * q + 2 * j + 1]);
        dg[8 * q + 2 * j] = h0 * u0 * d[2 * j];
        dg[8 * q + 2 * j + 1] = h1 * u1 * d[2 * j + 1];
        du[8 * q + 2 * j] = h0 * a[2 * j];
        du[8 * q + 2 * j + 1] = h1 * a[2 * j + 1];
      }
    }
    if (c + 32 < ncols) in = dgated_load(p, row, nc0 + 32);
    gated_store<BF16, NB, true>(dg, tmY, stg, scount, nc0, 0, wrow0, p.out_f32 != 0, p.N);
    gated_store<BF16, NB, true>(du, tmY, stg, scount, nc0, 1, wrow0, p.out_f32 != 0, p.N);
    if (p.dbias) {
      if (row >= p.T) {  // (0 x an infinite weight is no zero)
#pragma unroll
        for (int j = 0; j < 32; ++j) dg[j] = du[j] = 0.f;
      }
      warp_transpose_reduce32(dg);
      colp[c + lane] = dg[0];
      warp_transpose_reduce32(du);
      colp[gap + c + lane] = du[0];
    }
  }
}

// Column sums of a tile's 128 rows, the four lane quarters in order, into row
// `prow` of the partials (2N columns). cp: four times [dG: BN][dU: BN].
template <int BN, int NT>
__device__ __forceinline__ void dgated_write_partials(const TileParams& p, int prow, int n0, const float* cp, uint32_t et,
                                                      int ncols) {
  for (int c = et; c < 2 * ncols; c += NT) {
    const int half = c >= ncols ? 1 : 0, cc = c - half * ncols, n = n0 + cc;
    if (n >= p.N) continue;
    const float* s = cp + half * BN + cc;
    p.partials[(static_cast<int64_t>(prow) * 2 + half) * p.N + n] = ((s[0] + s[2 * BN]) + s[4 * BN]) + s[6 * BN];
  }
}

// As epi_finish_dbias, for both halves: the tile that takes a column block's
// last ticket adds the block's partial rows in ascending order (sixteen loads
// in flight) and resets the counter.
template <int NT>
__device__ __forceinline__ void dgated_finish_dbias(const TileParams& p, int nb, int n0, int rows, uint32_t et,
                                                    volatile int* flag, int ncols, int nblocks) {
  __threadfence();
  named_bar_sync(1, NT);
  if (et == 0) {
    int bits = 0;
    for (int b = 0; b < nblocks; ++b) {
      const int prev = atomicAdd(p.col_tickets + nb + b, rows);
      if (prev + rows == p.m_tiles) {
        p.col_tickets[nb + b] = 0;
        bits |= 1 << b;
      }
    }
    *flag = bits;
  }
  named_bar_sync(1, NT);
  const int bits = *flag;
  if (bits) {
    __threadfence();
    const int total = nblocks * ncols;
    for (int c = et; c < 2 * total; c += NT) {
      const int half = c >= total ? 1 : 0, cc = c - half * total, n = n0 + cc;
      if (!((bits >> (cc / ncols)) & 1) || n >= p.N) continue;
      const float* col = p.partials + static_cast<int64_t>(half) * p.N + n;
      const int64_t stride = 2 * static_cast<int64_t>(p.N);
      float s = 0.f;
      for (int m0 = 0; m0 < p.m_tiles; m0 += 16) {
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = m0 + j < p.m_tiles ? __ldcg(col + (m0 + j) * stride) : 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (m0 + j < p.m_tiles) s += x[j];
      }
      p.dbias[static_cast<int64_t>(half) * p.N + n] = s;
    }
  }
  named_bar_sync(1, NT);  // the flag word is reused by the next tile
}

}  // namespace ge
