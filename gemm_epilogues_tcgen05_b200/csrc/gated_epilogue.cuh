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

// The tiles of a CTA as a warp's DGatedStream walks them.
template <int BN>
struct TileSource {
  int tile, row;  // row: the warp's first of a tile
  __device__ __forceinline__ bool next(const TileParams& p, int& n0, int& ncols, int& row0) {
    if (tile >= p.num_tiles) return false;
    int mb, nb;
    tile_coords(tile, p.m_tiles, p.n_tiles, p.group_m, p.raster_n, mb, nb);
    tile += gridDim.x;
    n0 = nb * BN;
    ncols = BN;
    row0 = mb * kBM + row;
    return true;
  }
};

// Backward: an epilogue warp's own stream of G and U, in chunks of 32 rows x 32
// columns of both, in the order in which the warp will work on them and a slot or
// two before it does, across tiles: while a tile's products are still running its
// first chunks have come in. A slot holds [G, U][32 rows][64 bytes], 16-byte piece q of
// row r at q ^ ((r >> 1) & 3), so that a lane's own row and eight lanes' two rows
// are both free of bank conflicts; dG and dU take the places of G and U, and go out as
// 64 contiguous bytes of eight rows an instruction.
//
// Neither direction uses TMA: its rows of 64 bytes are as many requests as the
// operands' of 128, a quarter more in all, and the operands come late for them.
// T = K = 4096, N = 11008 (us): threads loading their own row's 64 bytes one chunk
// ahead and TMA stores 315; TMA both ways 294 (263 with the loads left out, 272
// without the stores).
template <class Source>
struct DGatedStream {
  const TileParams& p;
  uint32_t slots;   // shared address
  Source source;
  int n0 = 0, ncols = 0, row0 = 0, c = 0;  // the next chunk to be loaded
  bool live = true;
  uint32_t next_in = 0, next_out = 0;      // slots

  __device__ __forceinline__ DGatedStream(const TileParams& p_, const uint8_t* s, Source src)
      : p(p_), slots(smem_u32(s)), source(src) {}
  // piece lane % 4 of row 8 i + lane / 4
  static __device__ __forceinline__ uint32_t piece(int i) {
    const uint32_t row = 8 * i + (lane_id() >> 2);
    return row * 64 + (((lane_id() & 3u) ^ ((row >> 1) & 3u)) * 16);
  }
  __device__ __forceinline__ void issue() {
    while (live && (c >= ncols || n0 + c >= p.N)) {
      live = source.next(p, n0, ncols, row0);
      c = 0;
    }
    if (live) {
      const int col = n0 + c + 8 * static_cast<int>(lane_id() & 3u);
      const uint32_t dst = slots + next_in * 4096;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + 8 * i + static_cast<int>(lane_id() >> 2);
        const bool in = row < p.T && col < p.N;  // N is a multiple of 8
        const uint16_t* z = reinterpret_cast<const uint16_t*>(p.aux_in) + (in ? static_cast<int64_t>(row) * 2 * p.N + col : 0);
        cp_async_16(dst + piece(i), z, in);
        cp_async_16(dst + 2048 + piece(i), in ? z + p.N : z, in);
      }
      c += 32;
      next_in = next_in + 1 == kDGatedSlots ? 0 : next_in + 1;
    }
    cp_async_commit();
  }
  __device__ __forceinline__ void start() {
    for (int i = 0; i < kDGatedSlots; ++i) issue();
  }
  // the next chunk's slot, when it has come
  __device__ __forceinline__ uint32_t take() {
    cp_async_wait<kDGatedSlots - 1>();
    __syncwarp();
    const uint32_t at = slots + next_out * 4096;
    next_out = next_out + 1 == kDGatedSlots ? 0 : next_out + 1;
    return at;
  }
};

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

// fp32 outputs: 32 columns of one half through the slot, 128 bytes a row (piece q of
// row r at q ^ (r & 7)), 128 contiguous bytes of four rows an instruction.
__device__ __forceinline__ void dgated_store_f32(const TileParams& p, uint32_t slot, const float (&v)[32], int half,
                                                 int wrow0, int nc0) {
  const uint32_t lane = lane_id();
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q)
    st_shared_v4(slot + lane * 128 + ((q ^ (lane & 7u)) * 16),
                 make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                            __float_as_uint(v[4 * q + 3])));
  __syncwarp();
  const int col = nc0 + 4 * static_cast<int>(lane & 7u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t r = 4 * i + (lane >> 3);
    const int row = wrow0 + static_cast<int>(r);
    if (row < p.T && col < p.N)
      *reinterpret_cast<uint4*>(reinterpret_cast<float*>(p.out) + (static_cast<int64_t>(row) * 2 + half) * p.N + col) =
          ld_shared_v4(slot + r * 128 + (((lane & 7u) ^ (r & 7u)) * 16));
  }
}

// This warp's 32 rows from wrow0 on, columns n0 .. n0 + ncols - 1. With dbias, the
// column sums of the 32 rows go into a row of the partials of their own (2N
// columns), which dgated_dbias_kernel adds up.
template <bool BF16, class Stream>
__device__ __forceinline__ void dgated_rows(const TileParams& p, uint32_t tbase, int wrow0, int n0, int ncols, Stream& in) {
  const uint32_t lane = lane_id();
#pragma unroll 1
  for (int c = 0; c < ncols; c += 32) {
    const int nc0 = n0 + c;
    if (nc0 >= p.N) break;  // warp-uniform
    uint32_t r[32];
    tmem_ld_32x32b_x32(tbase + c, r);
    const uint32_t slot = in.take();
    const uint32_t own = slot + lane * 64, swz = ((lane >> 1) & 3u) * 16;
    tmem_wait_ld();
    float dg[32], du[32];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 ig = ld_shared_v4(own + ((q * 16) ^ swz)), iu = ld_shared_v4(own + 2048 + ((q * 16) ^ swz));
      const uint32_t wg[4] = {ig.x, ig.y, ig.z, ig.w};
      const uint32_t wu[4] = {iu.x, iu.y, iu.z, iu.w};
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
    if (p.out_f32) {
      dgated_store_f32(p, slot, dg, 0, wrow0, nc0);
      dgated_store_f32(p, slot, du, 1, wrow0, nc0);
    } else {
      // (a lane's row is read by that lane alone before it is replaced)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        st_shared_v4(own + ((q * 16) ^ swz),
                     make_uint4(pack2<BF16>(dg[8 * q], dg[8 * q + 1]), pack2<BF16>(dg[8 * q + 2], dg[8 * q + 3]),
                                pack2<BF16>(dg[8 * q + 4], dg[8 * q + 5]), pack2<BF16>(dg[8 * q + 6], dg[8 * q + 7])));
        st_shared_v4(own + 2048 + ((q * 16) ^ swz),
                     make_uint4(pack2<BF16>(du[8 * q], du[8 * q + 1]), pack2<BF16>(du[8 * q + 2], du[8 * q + 3]),
                                pack2<BF16>(du[8 * q + 4], du[8 * q + 5]), pack2<BF16>(du[8 * q + 6], du[8 * q + 7])));
      }
      __syncwarp();
      const int col = nc0 + 8 * static_cast<int>(lane & 3u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = wrow0 + 8 * i + static_cast<int>(lane >> 2);
        if (row < p.T && col < p.N) {
          uint16_t* z = reinterpret_cast<uint16_t*>(p.out) + static_cast<int64_t>(row) * 2 * p.N + col;
          *reinterpret_cast<uint4*>(z) = ld_shared_v4(slot + Stream::piece(i));
          *reinterpret_cast<uint4*>(z + p.N) = ld_shared_v4(slot + 2048 + Stream::piece(i));
        }
      }
    }
    __syncwarp();
    in.issue();
    if (p.dbias && wrow0 < p.T) {
      if (wrow0 + static_cast<int>(lane) >= p.T) {  // (0 x an infinite weight is no zero)
#pragma unroll
        for (int j = 0; j < 32; ++j) dg[j] = du[j] = 0.f;
      }
      warp_transpose_reduce32(dg);
      warp_transpose_reduce32(du);
      if (nc0 + static_cast<int>(lane) < p.N) {
        float* to = p.partials + static_cast<int64_t>(wrow0 >> 5) * 2 * p.N + nc0 + lane;
        to[0] = dg[0];
        to[p.N] = du[0];
      }
    }
  }
}

// The bias gradient: the partial sums' `rows` rows, in 8 runs of rows, each in
// ascending order, then the runs in order. 32 columns a block.
static __global__ void __launch_bounds__(256) dgated_dbias_kernel(const float* partials, int rows, int cols, float* dbias) {
  __shared__ float run[8][32];
  wait_for_inputs();
  const int n = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
  const int per = (rows + 7) / 8, r0 = y * per, r1 = min(rows, r0 + per);
  float s = 0.f;
  if (n < cols) {
    const float* at = partials + n;
    for (int r = r0; r < r1; r += 16) {
      float x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = r + j < r1 ? __ldcg(at + static_cast<int64_t>(r + j) * cols) : 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) s += x[j];
    }
  }
  run[y][threadIdx.x & 31] = s;
  __syncthreads();
  if (y == 0 && n < cols) {
#pragma unroll
    for (int j = 1; j < 8; ++j) s += run[j][threadIdx.x];
    dbias[n] = s;
  }
}

}  // namespace ge
