// grouped_kernel.cuh -- the linear-layer products grouped by expert: the rows
// of X are sorted by expert, expert e owns rows offsets[e] .. offsets[e+1]
// (any number of them, known only on the device) and its own weight.
//
//   forward / DRELU_BGRAD   Y[t][n] = epilog(sum_k X[t][k] W_e[k][n])
//   WGRAD                   dW_e[k][n] = sum over e's rows t of X[t][k] dZ[t][n]
//
// Swap-AB for every size: the features n are the MMA's M slot (128 per CTA,
// 256 per CTA pair) and the ragged dimension sits in the N slot, whose width
// is a field of the instruction descriptor -- a tile of 40 rows costs 64
// columns of MMA work, not 128 or 256, and no row of another expert is ever
// stored, because each accumulator column is one row and is stored or not on
// its own (a TMA store box cannot be clipped at an expert's last row). An
// expert's rows are cut into equal tiles of at most TR. WGRAD contracts over
// the ragged dimension instead; its N slot holds the k of dW.
//
// The tile list is made in the kernel: one warp of every CTA reads the
// offsets, and a prefix sum of each expert's tile count maps a tile index to
// its expert (binary search), so nothing is copied to the host, there is one
// launch, and a captured graph follows new offsets. Offsets are read as their
// running maximum cut to [0, T], so no value of them reaches outside X or Y.
//
// WGRAD's last k-block of an expert also loads rows of the next expert (or
// past the last one, where any bit pattern may stand). The MMA steps past the
// expert's rows are not issued, and within the last step of 16 the foreign
// rows are overwritten with zeros in both operands before it is issued: a
// zero in one operand alone would still let a NaN of the other through.
#pragma once

#include "skinny_kernel.cuh"
#include "tile2_kernel.cuh"

namespace ge {

constexpr int kMaxExperts = 1024;

struct GroupedParams {
  int32_t T, N, K, E;
  int32_t n_ft;             // feature tiles (of 128, CTA pairs 256)
  int32_t n_kt;             // WGRAD: k tiles of TR
  int32_t k_blocks;         // forward: stages of 64·KPS k
  int32_t group;            // row tiles per raster group
  int32_t aux_words;
  int32_t nfb;              // 128-feature blocks (DRELU_BGRAD tickets)
  const int32_t* offsets;   // E + 1
  const void* bias;         // E x N
  void* out;                // Y, dZ (T x N) or dW (E x K x N)
  uint32_t* aux_out;        // RELU_AUX_BIAS words; GELU_AUX_BIAS: T x N 16-bit Z
  const uint32_t* aux_in;
  float* dbias;             // DRELU_BGRAD: E x N
  float* partials;          // DRELU_BGRAD: [row tile][N]
  int* tickets;             // DRELU_BGRAD: [E][nfb], zero between launches
  int* status;
  uint64_t timeout_ns;
  int32_t bias_f32, out_f32;
  int32_t inject_stall;
  // one-CTA tiles, few of them: k split over several CTAs (grouped_splits)
  int32_t max_items;        // slots; 0: no split
  int32_t force_splits;     // override of grouped_splits' choice (0: none)
  float* split_slots;       // [max_items][TR / 4][128][4]
  int* split_tickets;       // [max_items], zero between launches
};

// Shared memory: a ring of stages (W: 128 features x 64·KPS k; X: this CTA's
// share of the row tile x 64·KPS k), the barriers and the tile table.
template <bool PAIR, int TR, int KPS>
struct GroupedSmem {
  static constexpr int BK = kBK * KPS;
  static constexpr int TRC = PAIR ? TR / 2 : TR;       // rows of the N slot held by this CTA
  static constexpr uint32_t A_CHUNK = 64 * BK * 2;     // MN-major: 64 features x BK
  static constexpr uint32_t A_SUB_MN = 64 * kBK * 2;   // MN-major: 64 k-rows of one chunk
  static constexpr uint32_t A_SUB_K = 128 * kBK * 2;   // K-major: 128 features x 64 k
  static constexpr uint32_t A_BYTES = 2 * A_CHUNK;
  static constexpr uint32_t B_SUB = TRC * kBK * 2;     // TRC rows x 64 k
  static constexpr uint32_t B_BYTES = KPS * B_SUB;
  static constexpr uint32_t STAGE = A_BYTES + B_BYTES;
  static constexpr uint32_t TABLE = 2 * (kMaxExperts + 1) * 4;
  static constexpr uint32_t FIXED = TABLE + 40 * 8 + 4 * 128 * 4 + 64 + 1024;
  static constexpr int STAGES = (232448 - FIXED) / STAGE > 10 ? 10 : (232448 - FIXED) / STAGE;
  static constexpr uint32_t OFF_A = 0;
  static constexpr uint32_t OFF_B = OFF_A + STAGES * A_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_B + STAGES * B_BYTES;
  static constexpr uint32_t N_BARS = 3 * STAGES + 5;   // full, empty, tail, tfull[2], tempty[2], drain
  static constexpr uint32_t OFF_MISC = OFF_BAR + 40 * 8;
  static constexpr uint32_t OFF_SUM = OFF_MISC + 64;   // DRELU_BGRAD: [2][warps per quarter][128] column sums
  static constexpr uint32_t OFF_TABLE = OFF_SUM + 4 * 128 * 4;
  static constexpr uint32_t BYTES = OFF_TABLE + TABLE + 1024;
  static_assert(N_BARS <= 40, "barrier space");
  static_assert(STAGES >= 3 && BYTES <= 232448, "grouped shared memory above the per-CTA limit");
};

// Epilogue warps: two per TMEM lane quarter (each every other chunk of 32
// rows) from 128-row tiles up, else one.
template <int TR>
struct GroupedEpiWarps {
  static constexpr int value = TR >= 128 ? 8 : 4;
};

// (The table's loops are not unrolled: it is the first code a launch runs, and
// fetching a longer one delayed the first load by 0.8 us.)
// start[i] for i in this lane's run [a, b): tiles of TR rows (times `mult`) of
// the experts before i.
template <int TR>
__device__ __forceinline__ void grouped_prefix(const GroupedParams& p, const int* offs, int* start, int mult, int a, int b) {
  const int lane = static_cast<int>(lane_id());
  int sum = 0;
#pragma unroll 1
  for (int i = a; i < b; ++i)
    if (i < p.E) sum += (offs[i + 1] - offs[i] + TR - 1) / TR;
  int s = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  s -= sum;  // tiles of the experts before this lane's
#pragma unroll 1
  for (int i = a; i < b; ++i) {
    start[i] = s * mult;
    if (i < p.E) s += (offs[i + 1] - offs[i] + TR - 1) / TR;
  }
}

// The expert table in shared memory, made by one warp: offs[0..E] (sanitised)
// and start[0..E], the first tile of each expert. Each lane takes a
// contiguous run of entries, so two warp scans do.
template <int TR>
__device__ __forceinline__ void grouped_table(const GroupedParams& p, int* offs, int* start, int tiles_per_mt) {
  const int lane = static_cast<int>(lane_id());
  if (p.E < 32) {
    // one entry a lane: both scans stay in registers (0.3 us less before the first load)
    int v = lane > p.E ? 0 : p.offsets ? max(0, min(p.offsets[lane], p.T)) : lane * p.T;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v = max(v, o);
    }
    const int after = __shfl_down_sync(0xffffffffu, v, 1);
    const int count = lane < p.E ? (after - v + TR - 1) / TR : 0;
    int s = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    if (lane <= p.E) {
      offs[lane] = v;
      start[lane] = (s - count) * tiles_per_mt;
    }
    __syncwarp();
    return;
  }
  const int per = (p.E + 1 + 31) / 32;
  const int a = min(lane * per, p.E + 1), b = min(a + per, p.E + 1);
  int mx = 0;
#pragma unroll 1
  for (int i = a; i < b; ++i) {
    mx = p.offsets ? max(mx, min(p.offsets[i], p.T)) : i * p.T;  // no offsets: one group of T rows
    offs[i] = mx;  // running maximum within the lane's run
  }
  int incl = mx;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl = max(incl, o);
  }
  int before = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) before = 0;
#pragma unroll 1
  for (int i = a; i < b; ++i) offs[i] = max(offs[i], before);
  __syncwarp();
  grouped_prefix<TR>(p, offs, start, tiles_per_mt, a, b);
}

// The estimated time (ns) of `tiles` tiles of `stages` stages, `rows` rows in
// the longest, each shared by s CTAs:
//   rounds of tiles x s work items x (stages / s x stage time + joining),
// where a stage's time is what one SM takes to stream it and joining is the
// partials' trip through L2 (write, ticket, read by the last to arrive),
// which grows with the parts and the rows. Fitted to measurements: T = 4, K =
// 8192, N = 512 takes 24.8 us unsplit and 16.7, 11.6, 9.7, 9.7 with 2, 4, 8, 16
// parts; T = 32, K = 4096, N = 1024 14.1 and 11.8, 9.6, 9.4, 11.0; WGRAD of 8192
// rows, K = N = 64 31.7 and 21.8, 15.9, 14.1, 15.6, K = N = 256 32.4 and 24.3,
// 19.4, 19.6, 32.0.
__host__ __device__ __forceinline__ int64_t grouped_split_ns(int tr, int64_t tiles, int s, int stages, int units, int rows) {
  const int64_t rounds = (tiles * s + units - 1) / units;
  const int r = rows < tr ? rows : tr;
  const int64_t join = s == 1 ? 0 : tr == 32 ? 2000 + s * (50 + r * 5) : 2600 + s * r * 8;
  return rounds * (static_cast<int64_t>((stages + s - 1) / s) * (tr == 32 ? 300 : 215) + join);
}

// May s CTAs share each tile? One item an SM at most (max_items slots), two
// stages each, and a contraction that is worth it at all.
__host__ __device__ __forceinline__ bool grouped_split_allowed(int64_t tiles, int s, int stages, int max_items) {
  return s == 1 || (tiles * s <= max_items && 2 * s <= stages && stages >= 16);
}

// How many CTAs share a tile's contraction when there are few tiles (few
// rows, few or narrow experts): the S up to 16 with the least estimated time.
// Every CTA computes the same from the same table.
template <int TR>
__device__ __forceinline__ int grouped_splits(const GroupedParams& p, int tiles, int stages, int units, int rows) {
  const int s = static_cast<int>(lane_id()) + 1;
  uint64_t cost = ~0ull;
  if (p.force_splits > 0) {
    if (s <= 16 && (s == 1 || static_cast<int64_t>(tiles) * s <= p.max_items))
      cost = static_cast<uint64_t>(abs(s - p.force_splits)) << 5 | static_cast<uint64_t>(s);
  } else if (s <= 16 && grouped_split_allowed(tiles, s, stages, p.max_items)) {
    cost = static_cast<uint64_t>(grouped_split_ns(TR, tiles, s, stages, units, rows)) << 5 | static_cast<uint64_t>(s);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, cost, d);
    cost = o < cost ? o : cost;
  }
  return static_cast<int>(cost & 31u);
}

// One output tile: features f0.., and `n` columns of the MMA's N slot of
// which the first `cols` are stored.
struct GroupedTile {
  int e;         // expert
  int f0;        // first feature of the (pair's) tile
  int c0;        // forward: first row of X; WGRAD: first k of dW
  int cols, n;   // stored columns; columns computed (a multiple of 32)
  int row0, rows;  // WGRAD: the expert's rows, the contraction
  int mt, mb;    // forward: the expert's row tiles and this tile's among them
};

template <int EPI, int TR, int FM>
__device__ __forceinline__ bool grouped_tile(const GroupedParams& p, const int* offs, const int* start, int tile,
                                             GroupedTile& w) {
  int mb, fb;
  if constexpr (EPI == EPI_WGRAD) {
    const int per = p.n_ft * p.n_kt;
    w.e = tile / per;
    if (w.e >= p.E) return false;
    tile_coords(tile - w.e * per, p.n_kt, p.n_ft, p.group, 0, mb, fb);
    w.c0 = mb * TR;
    w.cols = min(TR, p.K - w.c0);
    w.row0 = offs[w.e];
    w.rows = offs[w.e + 1] - w.row0;
    w.mt = 1;
    w.mb = mb;
  } else {
    if (tile >= start[p.E]) return false;
    int lo = 0, hi = p.E;  // start[lo] <= tile < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= tile)
        lo = mid;
      else
        hi = mid;
    }
    w.e = lo;
    w.row0 = offs[lo];
    w.rows = offs[lo + 1] - w.row0;
    w.mt = (w.rows + TR - 1) / TR;
    tile_coords(tile - start[lo], w.mt, p.n_ft, min(p.group, w.mt), 0, mb, fb);
    // equal tiles: since rows > (mt - 1) TR and a tile is at most TR, none is empty
    const int per = ((w.rows + w.mt - 1) / w.mt + 31) & ~31;
    w.c0 = w.row0 + mb * per;
    w.cols = min(per, w.rows - mb * per);
    w.mb = mb;
  }
  w.f0 = fb * FM;
  w.n = (w.cols + 31) & ~31;
  return true;
}

// 32 x 32 bits across the warp, transposed: lane l's bit j becomes lane j's bit
// l. Mask words are one per row, a lane of the epilogue holds one feature of 32
// rows. (One ballot or shuffle per row instead is a chain of 32 round trips:
// T = 3932, K = 192, N = 5824 took 36.5 us with the mask written so, 16.9 us
// without a mask.)
__device__ __forceinline__ uint32_t warp_transpose_bits(uint32_t x) {
  const uint32_t lane = lane_id();
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const uint32_t low = d == 16 ? 0x0000ffffu : d == 8 ? 0x00ff00ffu : d == 4 ? 0x0f0f0f0fu : d == 2 ? 0x33333333u : 0x55555555u;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, d);
    x = (lane & d) ? (x & ~low) | ((y >> d) & low) : (x & low) | ((y & low) << d);
  }
  return x;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// GELU(z) = z Phi(z) = max(z, 0) - |z| h(|z|) with h(a) = Phi(-a) = 2^q(a), so
// that the negative tail keeps its relative accuracy (an approximation of h
// itself, off by 2e-7 everywhere, was 0.2 % off at z = -4 and of the wrong sign
// at -5.2). q(a) = -1 + a (s(a) - a / (2 ln 2)): the Gaussian's exponent apart, s
// stays between -1.2 and -0.3, a polynomial of degree 14 in u = 2 a / 13 - 1
// (a weighted least-maximum fit on [0, 13], off by less than 2e-8 max(1, |q| / 2) /
// max(a, 0.3)), and the form is exact at a = 0. Measured over half a million
// points: |error| <= 9.3e-8 |z|, and relative to the result of a negative z at
// most 8e-7 down to -4, 2e-6 down to -6, 9e-6 down to -12.9, where h leaves the
// normal numbers and becomes 0 (ex2's flush); a is held at 13 beyond, so
// infinities give inf and 0, and max.NaN keeps NaN. Multiply-adds on two values an
// instruction and one ex2 each: with erff (an exponential and its branches) a 256
// x 256 tile's epilogue outlasted its products (microscaled T = 4096, N = 11008, K
// = 4096: 150 us, 96.5 with this, 74 without an activation; a polynomial for h
// took 92.3. E = 16, T = 1003, K = 2048, N = 5000: 23 us with either, 20.4 without).
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void gelu32(float (&v)[32]) {
  constexpr float kA = 13.0f, kS = 2.0f / 13.0f, kHalfLog2e = 0.72134752f;
  constexpr float kC[15] = {-0.47054109f, 0.258029431f, -0.160296753f, 0.102642007f, -0.0657589659f,
                            0.0410890728f, -0.0249870718f, 0.0165973958f, -0.00968039781f, -0.000120837707f,
                            0.00111253548f, 0.00610661181f, -0.00311078061f, -0.00396853918f, 0.00253350381f};
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float a0 = fminf(fabsf(v[j]), kA), a1 = fminf(fabsf(v[j + 1]), kA);
    const uint64_t a = pack_f32x2(a0, a1);
    const uint64_t u = fma_f32x2(a, pack_f32x2(kS, kS), pack_f32x2(-1.f, -1.f));
    uint64_t s = pack_f32x2(kC[14], kC[14]);
#pragma unroll
    for (int k = 13; k >= 0; --k) s = fma_f32x2(s, u, pack_f32x2(kC[k], kC[k]));
    s = fma_f32x2(a, pack_f32x2(-kHalfLog2e, -kHalfLog2e), s);
    const uint64_t q = fma_f32x2(a, s, pack_f32x2(-1.f, -1.f));
    float q0, q1, r0, r1;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(q0), "=f"(q1) : "l"(q));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r0) : "f"(v[j]));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r1) : "f"(v[j + 1]));
    v[j] = fmaf(-a0, exp2_ftz(q0), r0);
    v[j + 1] = fmaf(-a1, exp2_ftz(q1), r1);
  }
}

// Rows r .. r+3 of this lane's feature (a[0..3]) -> four features of one row:
// lane l ends with row r + (l & 3), features (l & ~3) .. + 3 of the warp's 32.
// Two exchanges (lanes l ^ 1, then l ^ 2). A warp then stores four rows with
// one instruction, 64 contiguous bytes (16-bit) or 128 (fp32) of each, instead
// of one row per instruction.
__device__ __forceinline__ void exchange4(float (&a)[4]) {
  const uint32_t lane = lane_id();
  const bool odd = (lane & 1u) != 0, hi = (lane & 2u) != 0;
  const float r0 = __shfl_xor_sync(0xffffffffu, odd ? a[0] : a[1], 1);
  const float r1 = __shfl_xor_sync(0xffffffffu, odd ? a[2] : a[3], 1);
  // even: rows 0 and 2, features l, l+1; odd: rows 1 and 3, features l-1, l
  const float p0 = odd ? r0 : a[0], p1 = odd ? a[1] : r0;
  const float q0 = odd ? r1 : a[2], q1 = odd ? a[3] : r1;
  const float s0 = __shfl_xor_sync(0xffffffffu, hi ? p0 : q0, 2);
  const float s1 = __shfl_xor_sync(0xffffffffu, hi ? p1 : q1, 2);
  a[0] = hi ? s0 : p0;
  a[1] = hi ? s1 : p1;
  a[2] = hi ? q0 : s0;
  a[3] = hi ? q1 : s1;
}

// The same for 16-bit results, given as two words of two rows each (p01 = rows
// r, r+1 of this lane's feature, p23 = rows r+2, r+3; the lower row in the low
// half): the halves change places between lanes l ^ 1, the words between l ^ 2.
__device__ __forceinline__ uint2 exchange4_16(uint32_t p01, uint32_t p23) {
  const uint32_t lane = lane_id();
  const bool hi = (lane & 2u) != 0;
  // even: (own low, other's low), odd: (other's high, own high)
  const uint32_t sel = (lane & 1u) ? 0x3276u : 0x5410u;
  const uint32_t p = __byte_perm(p01, __shfl_xor_sync(0xffffffffu, p01, 1), sel);
  const uint32_t q = __byte_perm(p23, __shfl_xor_sync(0xffffffffu, p23, 1), sel);
  const uint32_t s = __shfl_xor_sync(0xffffffffu, hi ? p : q, 2);
  return hi ? make_uint2(s, q) : make_uint2(p, s);
}

// Store 32 columns of the accumulator (this lane's feature, v[j] = row j of
// the chunk) into a row-major matrix of row length N: `base` is the address of
// (first row, the warp's first feature), `rows` the rows to store, `nvalid`
// the features of the warp below N (a multiple of 8, as N is).
// 16-bit: pk[j] holds rows 2j and 2j + 1.
__device__ __forceinline__ void store_packed16(const uint32_t (&pk)[16], void* base, int64_t N, int rows, int nvalid) {
  const int lane = static_cast<int>(lane_id());
  const int r = lane & 3, f = lane & ~3;
  uint16_t* dst = reinterpret_cast<uint16_t*>(base) + r * N + f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint2 w = exchange4_16(pk[2 * q], pk[2 * q + 1]);
    if (4 * q + r < rows && f < nvalid) *reinterpret_cast<uint2*>(dst) = w;
    dst += 4 * N;
  }
}

template <bool BF16>
__device__ __forceinline__ void store_cols16(const float (&v)[32], void* base, int64_t N, int rows, int nvalid) {
  uint32_t pk[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) pk[j] = pack2<BF16>(v[2 * j], v[2 * j + 1]);
  store_packed16(pk, base, N, rows, nvalid);
}

__device__ __forceinline__ void store_cols32(const float (&v)[32], void* base, int64_t N, int rows, int nvalid) {
  const int lane = static_cast<int>(lane_id());
  const int r = lane & 3, f = lane & ~3;
  float* dst = reinterpret_cast<float*>(base) + r * N + f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float a[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    exchange4(a);
    // evict first: fp32 results are large (weight gradients) and not read again
    // soon (E = 32 of 125 rows, K = 1024, N = 2048: 70.4 us without, 67.9 with)
    if (4 * q + r < rows && f < nvalid)
      __stcs(reinterpret_cast<float4*>(dst), make_float4(a[0], a[1], a[2], a[3]));
    dst += 4 * N;
  }
}

// Zero rows [r0, r1) of `chunks` MN-major operand chunks of 64 x 64 (128-byte
// rows; the swizzle moves 16-byte units only within a row), by one warp.
__device__ __forceinline__ void zero_rows(uint32_t addr, int chunks, int r0, int r1) {
  for (int c = 0; c < chunks; ++c)
    for (int x = r0 * 128 + static_cast<int>(lane_id()) * 16; x < r1 * 128; x += 512)
      st_shared_v4(addr + c * (64 * kBK * 2) + x, make_uint4(0u, 0u, 0u, 0u));
}

// Threads: producer and MMA warps, the epilogue's, and for WGRAD the warp that
// zeroes foreign rows, for DRELU_BGRAD the one that joins the column sums.
template <int EPI, int TR>
struct GroupedThreads {
  static constexpr int value = 64 + 32 * GroupedEpiWarps<TR>::value + (EPI == EPI_WGRAD || EPI == EPI_DRELU_BGRAD ? 32 : 0);
};

// SPLIT: an instance of its own for plans that may have few tiles (the joining
// code took registers from the epilogue of the others: WGRAD of 32 experts, K =
// 1024, N = 2048, 57 us without, 99 us with).
template <bool PAIR, int TR, int KPS, int EPI, bool BF16, bool WK, bool SPLIT = false>
__global__ void __launch_bounds__(GroupedThreads<EPI, TR>::value, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const GroupedParams p) {
  using L = GroupedSmem<PAIR, TR, KPS>;
  constexpr bool WG = EPI == EPI_WGRAD;
  static_assert(!SPLIT || !PAIR, "only one-CTA tiles are split");
  static_assert(!WG || (KPS == 1 && !WK && TR >= 128), "WGRAD stages one k-block of 64 rows");
  constexpr int STAGES = L::STAGES;
  constexpr int EW = GroupedEpiWarps<TR>::value;
  constexpr int ET = 32 * EW;
  constexpr int FM = PAIR ? 256 : 128;
  constexpr int BXR = L::TRC < 64 ? L::TRC : 64;  // rows per X box
  constexpr uint32_t TMEM_COLS = 2 * TR < 32 ? 32 : 2 * TR;
  constexpr uint32_t IDESC0 = idesc_f16(BF16, /*A MN-major*/ !WK, /*B MN-major*/ WG, FM, 0);
  constexpr uint16_t BOTH = 0x3;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem + L::OFF_A;
  uint8_t* sB = smem + L::OFF_B;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tailbar = empty + STAGES;
  uint64_t* tfull = tailbar + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  volatile int* sum_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 20);  // [2]
  volatile uint64_t* last_step = reinterpret_cast<volatile uint64_t*>(smem + L::OFF_MISC + 32);  // see wait_steps
  volatile int* split_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 12);
  int* split_count = reinterpret_cast<int*>(smem + L::OFF_MISC + 16);
  float* sums = reinterpret_cast<float*>(smem + L::OFF_SUM);
  int* offs = reinterpret_cast<int*>(smem + L::OFF_TABLE);
  int* start = offs + kMaxExperts + 1;

  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int unit = static_cast<int>(PAIR ? blockIdx.x >> 1 : blockIdx.x);
  const int units = static_cast<int>(PAIR ? gridDim.x >> 1 : gridDim.x);

  TileParams wp{};  // what the bounded wait reads
  wp.status = p.status;
  wp.timeout_ns = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], WG && PAIR ? 2 : 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tailbar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], PAIR ? 2 * EW : EW);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *last_step = globaltimer_ns();
    fence_barrier_init();
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, TMEM_COLS);
      tmem_relinquish();
    }
  }
  wait_for_inputs();
  if (warp == 2) {
    grouped_table<TR>(p, offs, start, p.n_ft);
    if constexpr (SPLIT) {
      __syncwarp();
      int most = 0;  // the longest expert
#pragma unroll 1
      for (int e = static_cast<int>(lane); e < p.E; e += 32) most = max(most, offs[e + 1] - offs[e]);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
      const int tiles = WG ? p.E * p.n_ft * p.n_kt : start[p.E];
      const int n = p.max_items > 0 && tiles > 0
                        ? grouped_splits<TR>(p, tiles, WG ? (most + kBK - 1) / kBK : p.k_blocks, units, WG ? p.K : most)
                        : 1;
      if (lane == 0) *split_count = n;
    }
  }
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();  // both CTAs' barriers exist before either side signals the other
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int S = SPLIT ? *split_count : 1;  // work item i: part i % S of tile i / S

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // (the whole warp walks the tiles, one elected lane issues: elect_one)
    const bool issuer = elect_one();
    uint32_t it = 0, s = 0, ph = 1;
    bool ok = true;
    const uint32_t full0 = PAIR ? mapa_shared(smem_u32(&full[0]), 0) : smem_u32(&full[0]);
    GroupedTile w;
    for (int item = unit; ok && grouped_tile<EPI, TR, FM>(p, offs, start, SPLIT ? item / S : item, w); item += units) {
      const int f0 = w.f0 + static_cast<int>(rank) * 128;
      const int nloc = PAIR ? w.n / 2 : w.n;
      const int c0 = w.c0 + static_cast<int>(rank) * nloc;
      const int kbs = WG ? (w.rows + kBK - 1) / kBK : p.k_blocks;
      const bool cut = WG && (w.rows & 15) != 0;  // the last k-block holds foreign rows within a step of 16
      const int part = SPLIT ? item % S : 0;
      const int kb0 = SPLIT ? kbs * part / S : 0, kb1 = SPLIT ? kbs * (part + 1) / S : kbs;
      // One-CTA forward tiles start at different k: started together, all CTAs
      // read the same columns of their weights at a time, which for rows of a
      // power-of-two length fall on few memory channels (E = 64, K = 1024, N =
      // 5000, N x K weights: 118.9 us with all at 0, 115.4 us; E = 8, K = 4096,
      // N = 11008: 112.5 and 109.7)
      const int rot = WG || PAIR || (SPLIT && S > 1) ? 0 : static_cast<int>(static_cast<uint32_t>(w.f0 / FM * 5 + w.e * 3) %
                                                               static_cast<uint32_t>(kbs));
      const int boxes = (nloc + (WG ? 64 : BXR) - 1) / (WG ? 64 : BXR);
      const uint32_t tx = L::A_BYTES + static_cast<uint32_t>(boxes) * (WG ? 64 * kBK * 2 : KPS * BXR * kBK * 2);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        ok = wait_steps(&empty[s], ph, wp, abort_flag, last_step, 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* a = sA + s * L::A_BYTES;
        uint8_t* b = sB + s * L::B_BYTES;
        if (issuer) {
          if (it % kStepStages == 0) *last_step = globaltimer_ns();
          if constexpr (WG) {
            const int t = w.row0 + kb * kBK;
            if (cut && kb == kbs - 1) {
              // signalled to this CTA's zeroing warp, which passes it on to the MMA
              mbar_arrive_expect_tx(&tailbar[s], tx);
              const uint32_t bar = smem_u32(&tailbar[s]);
              tma_load_3d<false>(a, &tmA, bar, f0, t, 0);
              tma_load_3d<false>(a + L::A_CHUNK, &tmA, bar, f0 + 64, t, 0);
              for (int i = 0; i < boxes; ++i) tma_load_3d<false>(b + i * (64 * kBK * 2), &tmB, bar, c0 + i * 64, t, 0);
            } else {
              if (rank == 0)
                mbar_arrive_expect_tx(&full[s], PAIR ? 2 * tx : tx);
              else
                mbar_arrive_peer(full0 + s * 8);
              const uint32_t bar = full0 + s * 8;
              tma_load_3d<PAIR>(a, &tmA, bar, f0, t, 0);
              tma_load_3d<PAIR>(a + L::A_CHUNK, &tmA, bar, f0 + 64, t, 0);
              for (int i = 0; i < boxes; ++i) tma_load_3d<PAIR>(b + i * (64 * kBK * 2), &tmB, bar, c0 + i * 64, t, 0);
            }
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&full[s], PAIR ? 2 * tx : tx);
            const uint32_t bar = full0 + s * 8;
            const int kr = kb + rot;
            const int k = (kr >= kbs ? kr - kbs : kr) * L::BK;
            if constexpr (WK) {
#pragma unroll
              for (int j = 0; j < KPS; ++j) tma_load_3d<PAIR>(a + j * L::A_SUB_K, &tmA, bar, k + j * kBK, f0, w.e);
            } else {
              tma_load_3d<PAIR>(a, &tmA, bar, f0, k, w.e);
              tma_load_3d<PAIR>(a + L::A_CHUNK, &tmA, bar, f0 + 64, k, w.e);
            }
#pragma unroll
            for (int j = 0; j < KPS; ++j)
              for (int i = 0; i < boxes; ++i)
                tma_load_3d<PAIR>(b + j * L::B_SUB + i * (BXR * kBK * 2), &tmB, bar, k + j * kBK, c0 + i * BXR, 0);
          }
        }
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // every issued copy has landed before the CTA can exit (in a pair the
    // leader's barriers count them: there the release by the MMA shows it)
    const uint32_t inflight = it < STAGES ? it : STAGES;
    for (uint32_t i = it - inflight; i < it; ++i)
      wait_steps(PAIR ? &empty[i % STAGES] : &full[i % STAGES], (i / STAGES) & 1u, wp, abort_flag, last_step, 2,
                   /*honour_abort=*/false);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    const bool issuer = elect_one();
    if (rank == 0) {
      uint32_t tcount = 0, s = 0, ph = 0;
      bool ok = true;
      GroupedTile w;
      for (int item = unit; ok && grouped_tile<EPI, TR, FM>(p, offs, start, SPLIT ? item / S : item, w); item += units) {
        const int kbs = WG ? (w.rows + kBK - 1) / kBK : p.k_blocks;
        const int part = SPLIT ? item % S : 0;
        const int kb0 = SPLIT ? kbs * part / S : 0, kb1 = SPLIT ? kbs * (part + 1) / S : kbs;
        if (kb0 == kb1) continue;  // nothing to contract (an expert without rows): the epilogue takes zeros
        const uint32_t buf = tcount & 1u;
        const uint32_t tph = (tcount >> 1) & 1u;
        ok = wait_steps(&tempty[buf], tph ^ 1u, wp, abort_flag, last_step, 3);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int tail = WG ? w.rows - (kbs - 1) * kBK : 0;  // rows in the last k-block
        const uint32_t idesc = IDESC0 | (static_cast<uint32_t>(w.n >> 3) << 17);
        const uint32_t d_tmem = tmem_base + buf * TR;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait_bounded(&full[s], ph, wp, abort_flag, 4);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const bool last = WG && kb == kbs - 1;
          // the peer's zeroed rows, acquired by a test of the phase that is
          // complete (a cluster-scope fence held every tile up by 1 us: E = 8 of
          // 1024 rows, K = 4096, N = 11008 551 us with it, 517 us without)
          if (PAIR && last && (w.rows & 15)) mbar_test_acquire_cluster(&full[s], ph);
          const uint32_t a0 = smem_u32(sA + s * L::A_BYTES);
          const uint32_t b0 = smem_u32(sB + s * L::B_BYTES);
          const int steps = last ? (tail + 15) / 16 : 4;
          if (issuer) {
#pragma unroll
            for (int j = 0; j < KPS; ++j) {
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) {
                // A MN-major: chunks A_CHUNK apart, 8 k-rows 1 KB apart, a step is 16 rows; K-major: 32 bytes a step
                const uint64_t ad = WK ? smem_desc_sw128(a0 + j * L::A_SUB_K + kk * 32, 16, 1024)
                                       : smem_desc_sw128(a0 + j * L::A_SUB_MN + kk * 2048, L::A_CHUNK, 1024);
                const uint64_t bd = WG ? smem_desc_sw128(b0 + kk * 2048, 64 * kBK * 2, 1024)
                                       : smem_desc_sw128(b0 + j * L::B_SUB + kk * 32, 16, 1024);
                const uint32_t acc = (kb > kb0 || j > 0 || kk > 0) ? 1u : 0u;
                if (!WG || kk < steps) {
                  if constexpr (PAIR)
                    umma_f16_pair(d_tmem, ad, bd, idesc, acc);
                  else
                    umma_f16(d_tmem, ad, bd, idesc, acc);
                }
              }
            }
            if constexpr (PAIR)
              umma_commit_pair(&empty[s], BOTH);
            else
              umma_commit(&empty[s]);
          }
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        // (fault injection: the epilogue then waits on a barrier nothing arrives on)
        if (issuer && !(p.inject_stall && tcount == 0 && (p.inject_stall == 1 || unit == 0))) {
          if constexpr (PAIR)
            umma_commit_pair(&tfull[buf], BOTH);
          else
            umma_commit(&tfull[buf]);
        }
        ++tcount;
      }
      if (issuer) {
        if constexpr (PAIR)
          umma_commit_pair(drain, BOTH);
        else
          umma_commit(drain);
      }
    }
    // every MMA that writes this CTA's tensor memory is done before it is freed
    wait_steps(drain, 0, wp, abort_flag, last_step, 5, /*honour_abort=*/false);
    __syncwarp();
  } else if (WG && warp == 2 + EW) {
    // ---------------------------------------------- foreign rows (WGRAD)
    // Ahead of the MMA by the depth of the ring: waits for the copies of an
    // expert's last k-block in this CTA, zeroes the foreign rows of its last
    // step and counts the stage in for the MMA.
    if constexpr (WG) {
      uint32_t it = 0, phases = 0;  // one phase bit per stage
      bool ok = true;
      const uint32_t full0 = PAIR ? mapa_shared(smem_u32(&full[0]), 0) : smem_u32(&full[0]);
      GroupedTile w;
      for (int item = unit; ok && grouped_tile<EPI, TR, FM>(p, offs, start, SPLIT ? item / S : item, w); item += units) {
        const int kbs = (w.rows + kBK - 1) / kBK;
        const int part = SPLIT ? item % S : 0;
        const int kb0 = SPLIT ? kbs * part / S : 0, kb1 = SPLIT ? kbs * (part + 1) / S : kbs;
        it += static_cast<uint32_t>(kb1 - kb0);
        if ((w.rows & 15) == 0 || kb1 == kb0 || kb1 < kbs) continue;
        const uint32_t s = (it - 1) % STAGES;
        ok = wait_steps(&tailbar[s], (phases >> s) & 1u, wp, abort_flag, last_step, 9);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        phases ^= 1u << s;
        const int tail = w.rows & (kBK - 1);
        const int r1 = (tail + 15) & ~15;
        zero_rows(smem_u32(sA) + s * L::A_BYTES, 2, tail, r1);
        zero_rows(smem_u32(sB) + s * L::B_BYTES, ((PAIR ? w.n / 2 : w.n) + 63) / 64, tail, r1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_cluster(full0 + s * 8);
          else
            mbar_arrive(&full[s]);
        }
      }
    }
  } else if (EPI == EPI_DRELU_BGRAD && warp == 2 + EW) {
    // ------------------------------------------------- column sums (DRELU_BGRAD)
    // A tile's sums over its rows, the quarter's warps in order, straight to
    // dbias or (an expert of several row tiles) to one partial row per tile;
    // the block of features' last tile adds those in tile order, so the result
    // does not depend on timing. In a warp of its own: the fence before the
    // ticket waits for its few stores only, not for the epilogue's.
    if constexpr (EPI == EPI_DRELU_BGRAD) {
      uint32_t dcount = 0;
      GroupedTile w;
      for (int item = unit; grouped_tile<EPI, TR, FM>(p, offs, start, SPLIT ? item / S : item, w); item += units, ++dcount) {
        const uint32_t b = dcount & 1u;
        named_bar_sync(2 + b, ET + 32);
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i] = sums[b * (EW / 4) * 128 + i * 32 + lane];
          if constexpr (EW == 8) s[i] += sums[(b * 2 + 1) * 128 + i * 32 + lane];
        }
        // (after an abort the sums are not whole; one lane's view, so that all agree)
        const bool use = __shfl_sync(0xffffffffu, sum_flag[b] != 0 && *abort_flag == 0 ? 1 : 0, 0) != 0;
        named_bar_arrive(4 + b, ET + 32);
        const int n0 = w.f0 + static_cast<int>(rank * 128u + lane);
        if (!use || w.f0 + static_cast<int>(rank) * 128 >= p.N) continue;  // warp-uniform
        float* out = p.dbias + static_cast<int64_t>(w.e) * p.N;
        if (w.mt > 1) {
          const int64_t mrow = start[w.e] / p.n_ft;
          float* row = p.partials + (mrow + w.mb) * p.N;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n0 + i * 32 < p.N) row[n0 + i * 32] = s[i];
          __threadfence();
          __syncwarp();
          int last = 0;
          if (lane == 0) {
            int* tk = p.tickets + static_cast<int64_t>(w.e) * p.nfb + (w.f0 >> 7) + static_cast<int>(rank);
            last = atomicAdd(tk, 1) == w.mt - 1;
            if (last) *tk = 0;  // ready for the next launch
          }
          if (__shfl_sync(0xffffffffu, last, 0) == 0) continue;
          __threadfence();
          const float* src = p.partials + mrow * p.N;
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = 0.f;
          for (int m0 = 0; m0 < w.mt; m0 += 8) {
            float x[8][4];
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[m][i] = m0 + m < w.mt && n0 + i * 32 < p.N ? __ldcg(src + static_cast<int64_t>(m0 + m) * p.N + n0 + i * 32) : 0.f;
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[i] += x[m][i];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i * 32 < p.N) out[n0 + i * 32] = s[i];
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t ew = warp & 3u;         // TMEM lane quarter
    const uint32_t eh = (warp - 2u) >> 2;  // which of the quarter's warps
    const uint32_t et = threadIdx.x - 64;
    uint32_t tcount = 0, dcount = 0;
    bool ok = true;
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&tempty[0]), 0) : smem_u32(&tempty[0]);
    if constexpr (EPI == EPI_DRELU_BGRAD) {
      // experts without rows: no tile of theirs exists, and their bias gradient is zero
      for (int e = static_cast<int>(blockIdx.x); e < p.E; e += static_cast<int>(gridDim.x))
        if (offs[e] == offs[e + 1]) {
          for (int n = static_cast<int>(et); n < p.N; n += ET) p.dbias[static_cast<int64_t>(e) * p.N + n] = 0.f;
          if (et == 0) *last_step = globaltimer_ns();
        }
    }
    GroupedTile w;
    for (int item = unit; grouped_tile<EPI, TR, FM>(p, offs, start, SPLIT ? item / S : item, w); item += units) {
      const int fw = w.f0 + static_cast<int>(rank * 128u + ew * 32u);  // the warp's first feature
      const int n = fw + static_cast<int>(lane);
      const bool n_ok = n < p.N;
      const int nvalid = max(0, min(32, p.N - fw));
      const int word = fw >> 5;
      const int kbs = WG ? (w.rows + kBK - 1) / kBK : p.k_blocks;
      const int part = SPLIT ? item % S : 0;
      const bool empty_tile = SPLIT ? kbs * part / S == kbs * (part + 1) / S : kbs == 0;
      bool finisher = true;  // of a split tile, the CTA that takes its last ticket
      const uint32_t buf = tcount & 1u;
      const uint32_t tph = (tcount >> 1) & 1u;
      float bias_n = 0.f;
      if constexpr (AddsBias<EPI>::value)
        if (n_ok) bias_n = load_bias<BF16>(p.bias, p.bias_f32, static_cast<int64_t>(w.e) * p.N + n);
      float dsum = 0.f;
      // DRELU_BGRAD: the first chunk's mask words, loaded before the accumulator wait
      uint32_t mnext = 0u;
      const auto mask_word = [&](int c) -> uint32_t {
        const int r = c * 32 + static_cast<int>(lane);
        return (r < w.cols && word < p.aux_words)
                   ? __ldg(p.aux_in + static_cast<int64_t>(w.c0 + r) * p.aux_words + word)
                   : 0u;
      };
      if constexpr (EPI == EPI_DRELU_BGRAD)
        if (!SPLIT || S == 1) mnext = mask_word(static_cast<int>(eh));
      if (!empty_tile) {
        if (ok) ok = wait_steps(&tfull[buf], tph, wp, abort_flag, last_step, 6);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
      {
        const uint32_t tbase = tmem_base + ((ew * 32u) << 16) + buf * TR;
        const int64_t orow = WG ? static_cast<int64_t>(w.e) * p.K + w.c0 : static_cast<int64_t>(w.c0);
        constexpr int STEP = EW / 4;  // the quarter's warps take chunks of 32 columns in turn
        const auto finish = [&](const uint32_t (&acc)[32], int c, bool joined = false) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = empty_tile && !joined ? 0.f : __uint_as_float(acc[j]);
          const int rows = w.cols - c * 32;
          const int64_t at = (orow + c * 32) * p.N + fw;
          if constexpr (EPI == EPI_DRELU_BGRAD) {
            const uint32_t mine = warp_transpose_bits(mnext);  // bit j: this feature of row j
            if ((c + STEP) * 32 < w.n) mnext = mask_word(c + STEP);
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              v[j] = (mine >> j) & 1u ? v[j] : 0.f;
              part[j & 3] += v[j];  // rows past the tile have no mask bit set
            }
            dsum += (part[0] + part[1]) + (part[2] + part[3]);
          } else if constexpr (!PlainStore<EPI>::value) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += bias_n;
            if constexpr (EPI == EPI_GELU_AUX_BIAS)
              store_cols16<BF16>(v, reinterpret_cast<uint16_t*>(p.aux_out) + at, p.N, rows, nvalid);
            if constexpr (AppliesGelu<EPI>::value) gelu32(v);
            if constexpr (EPI == EPI_RELU_BIAS || EPI == EPI_RELU_AUX_BIAS) {
              uint32_t bits = 0u;  // of this feature, by row
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const bool pos = v[j] > 0.f;
                if constexpr (EPI == EPI_RELU_AUX_BIAS) bits |= (pos ? 1u : 0u) << j;
                v[j] = pos ? v[j] : 0.f;
              }
              if constexpr (EPI == EPI_RELU_AUX_BIAS) {
                const uint32_t mine = warp_transpose_bits(n_ok ? bits : 0u);
                if (static_cast<int>(lane) < rows && word < p.aux_words)
                  p.aux_out[(orow + c * 32 + static_cast<int>(lane)) * p.aux_words + word] = mine;
              }
            }
          }
          if (p.out_f32)
            store_cols32(v, reinterpret_cast<float*>(p.out) + at, p.N, rows, nvalid);
          else
            store_cols16<BF16>(v, reinterpret_cast<uint16_t*>(p.out) + at, p.N, rows, nvalid);
        };
        if (SPLIT && S > 1 && ok) {
          // a part of a split tile: leave the fp32 accumulator in this item's slot,
          // four rows of a feature together (16-byte stores and loads)
          float4* slot = reinterpret_cast<float4*>(p.split_slots) + static_cast<int64_t>(item) * (TR * 32) + ew * 32 + lane;
#pragma unroll 1
          for (int c = static_cast<int>(eh); c * 32 < w.cols; c += STEP) {
            uint32_t r[32];
            if (!empty_tile) {
              tmem_ld_32x32b_x32(tbase + c * 32, r);
              tmem_wait_ld();
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (c * 32 + 4 * q < w.cols)
                slot[(c * 8 + q) * 128] = empty_tile ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                     : make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                                                                   __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
          }
          if (!empty_tile) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
        }
        // two chunks are read together, and the accumulator is handed back as
        // soon as the last of them is in registers, before it is stored
#pragma unroll 1
        for (int c = static_cast<int>(eh); ok && (!SPLIT || S == 1) && (c * 32 < w.n || c == static_cast<int>(eh)); c += 2 * STEP) {
          const bool one = c * 32 < w.n, two = (c + STEP) * 32 < w.n;
          uint32_t r0[32], r1[32];
          if (!empty_tile) {
            if (one) tmem_ld_32x32b_x32(tbase + c * 32, r0);
            if (two) tmem_ld_32x32b_x32(tbase + (c + STEP) * 32, r1);
            tmem_wait_ld();
            if ((c + 2 * STEP) * 32 >= w.n) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if constexpr (PAIR)
                  mbar_arrive_peer(tempty0 + buf * 8);
                else
                  mbar_arrive(&tempty[buf]);
              }
            }
          }
          if (one) finish(r0, c);
          if (two) finish(r1, c + STEP);
        }
        if (SPLIT && S > 1) {
          const int tile = item / S;
          __threadfence();
          named_bar_sync(1, ET);
          if (et == 0) {
            const int last = ok && atomicAdd(p.split_tickets + tile, 1) == S - 1;
            if (last) p.split_tickets[tile] = 0;  // ready for the next launch
            *split_flag = last;
          }
          named_bar_sync(1, ET);  // (met by every warp, also after a wait that ran out)
          finisher = *split_flag != 0;
          if (finisher && ok) {
            // the parts in order, so the sum does not depend on who came last;
            // SB parts' loads of a chunk are in flight together
            __threadfence();
            constexpr int SB = EW == 4 ? 4 : 2;
            const float4* base = reinterpret_cast<const float4*>(p.split_slots) +
                                 static_cast<int64_t>(tile) * S * (TR * 32) + ew * 32 + lane;
            if constexpr (EPI == EPI_DRELU_BGRAD) mnext = mask_word(static_cast<int>(eh));
#pragma unroll 1
            for (int c = static_cast<int>(eh); c * 32 < w.cols; c += STEP) {
              float sum[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) sum[j] = 0.f;
#pragma unroll 1
              for (int s0 = 0; s0 < S; s0 += SB) {
                float4 x[SB][8];
#pragma unroll
                for (int s = 0; s < SB; ++s)
#pragma unroll
                  for (int q = 0; q < 8; ++q)
                    x[s][q] = s0 + s < S && c * 32 + 4 * q < w.cols
                                  ? __ldcg(base + static_cast<int64_t>(s0 + s) * (TR * 32) + (c * 8 + q) * 128)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int s = 0; s < SB; ++s)
#pragma unroll
                  for (int q = 0; q < 8; ++q) {
                    sum[4 * q] += x[s][q].x;
                    sum[4 * q + 1] += x[s][q].y;
                    sum[4 * q + 2] += x[s][q].z;
                    sum[4 * q + 3] += x[s][q].w;
                  }
              }
              uint32_t r[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(sum[j]);
              finish(r, c, true);
            }
          }
        }
      }
      if (!empty_tile)
        ++tcount;
      else if (et == 0)
        *last_step = globaltimer_ns();
      if constexpr (EPI == EPI_DRELU_BGRAD) {
        // this tile's column sums to the joining warp, two tiles deep
        const uint32_t b = dcount & 1u;
        if (dcount >= 2) named_bar_sync(4 + b, ET + 32);  // it has read the ones before
        sums[(b * (EW / 4) + eh) * 128 + ew * 32 + lane] = dsum;
        if (et == 0) sum_flag[b] = finisher ? 1 : 0;
        named_bar_arrive(2 + b, ET + 32);
        ++dcount;
      }
    }
    if constexpr (EPI == EPI_DRELU_BGRAD)
      for (uint32_t i = dcount < 2 ? 0 : dcount - 2; i < dcount; ++i) named_bar_sync(4 + (i & 1u), ET + 32);
  }

  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();  // neither CTA leaves while the other may still signal it
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, TMEM_COLS);
    else
      tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// Column sums of X per expert (WGRAD's optional bias gradient), one read of X.
// A block takes 256 columns of one expert and one of `slices` equal parts of
// its rows (more than one where experts x columns alone would not fill the
// GPU); its 8 warps stride over the rows, 16 bytes a lane. Warps are added in
// order, and the block that takes a (columns, expert)'s last ticket adds the
// slices in order, so the sum does not depend on timing.
template <bool BF16>
__global__ void __launch_bounds__(256) grouped_colsum_kernel(const uint16_t* __restrict__ X, const int32_t* offsets, int T,
                                                             int E, int K, int slices, float* partials, int* tickets,
                                                             float* __restrict__ dbias) {
  __shared__ float part[8][256];
  __shared__ int span[2];
  __shared__ int last;
  wait_for_inputs();
  const int e = blockIdx.y, z = blockIdx.z;
  const int lane = static_cast<int>(lane_id()), r = static_cast<int>(threadIdx.x >> 5);
  if (threadIdx.x < 32) {  // offsets as the products read them: the running maximum cut to [0, T]
    int m = 0, at_e = 0;
    for (int i = lane; i <= e + 1; i += 32) {
      m = max(m, min(offsets[i], T));
      if (i <= e) at_e = m;
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      at_e = max(at_e, __shfl_xor_sync(0xffffffffu, at_e, d));
    }
    if (lane == 0) {
      const int64_t n = m - at_e;
      span[0] = at_e + static_cast<int>(n * z / slices);
      span[1] = at_e + static_cast<int>(n * (z + 1) / slices);
    }
  }
  __syncthreads();
  const int k = blockIdx.x * 256 + lane * 8;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (k < K) {
    const auto add = [&](uint4 v) {
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (BF16)
          f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]));
        else
          f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        s[2 * i] += f.x;
        s[2 * i + 1] += f.y;
      }
    };
    int t = span[0] + r;
    for (; t + 24 < span[1]; t += 32) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(X + static_cast<int64_t>(t + 8 * i) * K + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) add(v[i]);
    }
    for (; t < span[1]; t += 8) add(*reinterpret_cast<const uint4*>(X + static_cast<int64_t>(t) * K + k));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[r][lane * 8 + i] = s[i];
  __syncthreads();
  const int kc = blockIdx.x * 256 + static_cast<int>(threadIdx.x);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += part[i][threadIdx.x];
  const int64_t at = static_cast<int64_t>(e) * K + kc;
  if (slices == 1) {
    if (kc < K) dbias[at] = sum;
    return;
  }
  const int64_t stride = static_cast<int64_t>(E) * K;
  if (kc < K) partials[z * stride + at] = sum;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    int* tk = tickets + static_cast<int64_t>(e) * gridDim.x + blockIdx.x;
    last = atomicAdd(tk, 1) == slices - 1;
    if (last) *tk = 0;  // ready for the next launch
  }
  __syncthreads();
  if (last && kc < K) {
    __threadfence();
    float t = 0.f;
    for (int i0 = 0; i0 < slices; i0 += 16) {  // sixteen loads in flight (8192 rows, K = 256, 64 slices: 9.2 to 6.4 us)
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i0 + i < slices ? __ldcg(partials + (i0 + i) * stride + at) : 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) t += x[i];
    }
    dbias[at] = t;
  }
}

}  // namespace ge
