// mx_kernel.cuh -- the product of two microscaled 4-bit operands,
//   Y[t][n] = epilog(sum_k X[t][k] W[n][k]),
// both held as e2m1 values with a power-of-two scale per 32 elements of k
// (mx_quant.cuh), for one weight or grouped by expert.
//
// Roles, tiles and epilogue are the grouped kernel's (grouped_kernel.cuh): the
// features are the MMA's M slot, the rows its N slot. What differs:
//   * tcgen05.mma kind::mxf4 multiplies 64 k a step and applies the scales
//     itself: sum over blocks of (scale_a scale_b) (sum of 32 products), fp32
//     accumulation. It reads the scales from tensor memory, one 32-bit column
//     holding 4 consecutive blocks of a row, row r in lane r % 32 (repeated in
//     all four lane quarters) of column r / 32.
//   * a stage is 256 k: 128 bytes a row, the same bytes as 64 k of a 16-bit
//     operand for four times the products, so the same ring feeds it. Its
//     scales (2 tiles of 512 bytes per 128 rows) come with it and are copied
//     to tensor memory (tcgen05.cp 32x128b.warpx4) by the thread that issues
//     the MMAs, which keeps the two in order; alternate stages use alternate
//     columns.
//   * CTA pairs compute 256 x 256, whose accumulator and the scales do not fit
//     twice in the 512 columns. One accumulator, then: eight epilogue warps
//     bring it to registers (rounded and packed to 16 bits as they read it) and
//     hand it back, so the next tile's MMAs wait for that drain only, not for
//     the stores.
#pragma once

#include "grouped_kernel.cuh"

namespace ge {

struct MxParams {
  GroupedParams g;
  int32_t wt;  // scale tiles (128 features) of one weight
};

template <bool PAIR, int TR>
struct MxSmem {
  static constexpr int BK = 256;                        // k per stage: 128 bytes a row
  static constexpr int TRC = PAIR ? TR / 2 : TR;
  static constexpr int RA = TR / 128;                   // scale tiles along the rows
  static constexpr uint32_t A_BYTES = 128 * 128;
  static constexpr uint32_t B_BYTES = TRC * 128;
  static constexpr uint32_t SF_TILE = 1024;             // 128 rows x 8 blocks
  static constexpr uint32_t SF_BYTES = (1 + RA) * SF_TILE;
  static constexpr uint32_t STAGE = A_BYTES + B_BYTES + SF_BYTES;
  static constexpr uint32_t TABLE = 3 * (kMaxExperts + 1) * 4;
  static constexpr uint32_t FIXED = TABLE + 32 * 8 + 64 + 1024;
  static constexpr int STAGES = (232448 - FIXED) / STAGE;
  static constexpr uint32_t OFF_A = 0;
  static constexpr uint32_t OFF_B = OFF_A + STAGES * A_BYTES;
  static constexpr uint32_t OFF_SF = OFF_B + STAGES * B_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_SF + STAGES * SF_BYTES;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 32 * 8;
  static constexpr uint32_t OFF_TABLE = OFF_MISC + 64;
  static constexpr uint32_t BYTES = OFF_TABLE + TABLE + 1024;
  static_assert(2 * STAGES + 5 <= 32 && STAGES >= 4 && BYTES <= 232448, "microscaled ring");
};

// Instruction descriptor of kind::mxf4: scale byte pair of B in [4,6), A and B
// format in [7,10) and [10,12) (1 = e2m1), both K-major, N >> 3 in [17,23),
// scale type at 23 (1 = e8m0), M >> 7 in [27,29), scale byte pair of A in
// [29,31), K = 64 (bit 31 clear).
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 7) << 27);
}

template <bool PAIR>
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// One scale tile (32 lanes x 16 bytes) from shared memory to four columns of
// tensor memory, repeated in the four lane quarters; with PAIR in both CTAs,
// each from its own shared memory.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  // no swizzle; 8-row core matrices of 16-byte rows, 128 bytes apart
  const uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1u) << 16) |
                     (static_cast<uint64_t>(128u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46);
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

struct MxTile {
  int e, f0, c0, cols, n;
  int srow;  // scale tile of the first row
};

// One-CTA tiles start at different k, as the grouped kernel's do: with all
// CTAs at the same columns of rows of K / 2 bytes, few memory channels are
// asked at a time.
template <bool PAIR>
__device__ __forceinline__ int mx_first_k(const MxTile& w, int k_blocks) {
  return PAIR ? 0 : static_cast<int>(static_cast<uint32_t>(w.f0 / 128 * 5 + w.e * 3) % static_cast<uint32_t>(k_blocks));
}

template <int TR, int FM>
__device__ __forceinline__ bool mx_tile(const GroupedParams& p, const int* offs, const int* start, const int* stile,
                                        int tile, MxTile& w) {
  if (tile >= start[p.E]) return false;
  int lo = 0, hi = p.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= tile)
      lo = mid;
    else
      hi = mid;
  }
  const int rows = offs[lo + 1] - offs[lo];
  const int mt = (rows + TR - 1) / TR;
  int mb, fb;
  tile_coords(tile - start[lo], mt, p.n_ft, min(p.group, mt), 0, mb, fb);
  w.e = lo;
  w.f0 = fb * FM;
  w.c0 = offs[lo] + mb * TR;
  w.cols = min(TR, rows - mb * TR);
  w.n = (w.cols + 31) & ~31;
  w.srow = stile[lo] + mb * (TR / 128);
  return true;
}

template <bool PAIR, int TR, int EPI, bool BF16, bool F32>
__global__ void __launch_bounds__(320, 1)
    mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB, const MxParams mp) {
  using L = MxSmem<PAIR, TR>;
  const GroupedParams& p = mp.g;
  constexpr int STAGES = L::STAGES;
  constexpr int EW = 8;
  constexpr int FM = PAIR ? 256 : 128;
  constexpr int BXR = PAIR ? 64 : 32;
  constexpr int DBUF = PAIR ? 1 : 2;         // accumulators
  constexpr uint32_t SF_COL = 256;           // scales: two sets of (8 + 8 RA) columns
  constexpr uint32_t SF_SET = 8 + 8 * L::RA;
  static_assert(DBUF * TR <= 256 && SF_COL + 2 * SF_SET <= 512, "tensor memory");
  constexpr uint32_t IDESC0 = idesc_mxf4(FM, 0);
  constexpr uint16_t BOTH = 0x3;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem + L::OFF_A;
  uint8_t* sB = smem + L::OFF_B;
  uint8_t* sSF = smem + L::OFF_SF;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  volatile uint64_t* last_step = reinterpret_cast<volatile uint64_t*>(smem + L::OFF_MISC + 8);  // see wait_steps
  int* offs = reinterpret_cast<int*>(smem + L::OFF_TABLE);
  int* start = offs + kMaxExperts + 1;
  int* stile = start + kMaxExperts + 1;  // first scale tile (128 rows) of each expert

  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int unit = static_cast<int>(PAIR ? blockIdx.x >> 1 : blockIdx.x);
  const int units = static_cast<int>(PAIR ? gridDim.x >> 1 : gridDim.x);
  TileParams wp{};
  wp.status = p.status;
  wp.timeout_ns = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
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
    prefetch_tensormap(&tmSA);
    prefetch_tensormap(&tmSB);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  wait_for_inputs();
  if (warp == 2) {
    grouped_table<TR>(p, offs, start, p.n_ft);
    const int per = (p.E + 1 + 31) / 32;
    const int a = min(static_cast<int>(lane) * per, p.E + 1);
    grouped_prefix<128>(p, offs, stile, 1, a, min(a + per, p.E + 1));
  }
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();  // both CTAs' barriers exist before either side signals the other
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // (the whole warp walks the tiles, one elected lane issues: elect_one)
    const bool issuer = elect_one();
    uint32_t it = 0, s = 0, ph = 1;
    bool ok = true;
    const uint32_t full0 = PAIR ? mapa_shared(smem_u32(&full[0]), 0) : smem_u32(&full[0]);
    MxTile w;
    for (int tile = unit; ok && mx_tile<TR, FM>(p, offs, start, stile, tile, w); tile += units) {
      const int f0 = w.f0 + static_cast<int>(rank) * 128;
      const int nloc = PAIR ? w.n / 2 : w.n;
      const int c0 = w.c0 + static_cast<int>(rank) * nloc;
      const int boxes = (nloc + BXR - 1) / BXR;
      const int ra = (w.cols + 127) / 128;  // scale tiles along the rows; both CTAs of a pair need all of them
      // a peer whose features are all past N loads its scales at a tile past the last (zeros)
      const int wtile = f0 < p.N ? w.e * mp.wt + f0 / 128 : p.E * mp.wt;
      const uint32_t tx = (PAIR ? 2u : 1u) * (L::A_BYTES + static_cast<uint32_t>(boxes) * BXR * 128 +
                                              static_cast<uint32_t>(1 + ra) * L::SF_TILE);
      int kb = mx_first_k<PAIR>(w, p.k_blocks);
      for (int i_k = 0; i_k < p.k_blocks; ++i_k, ++it, kb = kb + 1 == p.k_blocks ? 0 : kb + 1) {
        ok = wait_bounded(&empty[s], ph, wp, abort_flag, 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (issuer) {
          if (PAIR && it % kStepStages == 0) *last_step = globaltimer_ns();
          if (rank == 0) mbar_arrive_expect_tx(&full[s], tx);
          const uint32_t bar = full0 + s * 8;
          uint8_t* sf = sSF + s * L::SF_BYTES;
          tma_load_3d<PAIR>(sA + s * L::A_BYTES, &tmA, bar, kb * 128, f0, w.e);
          for (int i = 0; i < boxes; ++i)
            tma_load_3d<PAIR>(sB + s * L::B_BYTES + i * (BXR * 128), &tmB, bar, kb * 128, c0 + i * BXR, 0);
          tma_load_3d<PAIR>(sf, &tmSA, bar, 0, kb * 2, wtile);
          tma_load_3d<PAIR>(sf + L::SF_TILE, &tmSB, bar, 0, kb * 2, w.srow);
          if (L::RA == 2 && ra == 2) tma_load_3d<PAIR>(sf + 2 * L::SF_TILE, &tmSB, bar, 0, kb * 2, w.srow + 1);
        }
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    const uint32_t inflight = it < STAGES ? it : STAGES;
    for (uint32_t i = it - inflight; i < it; ++i)
      wait_bounded(PAIR ? &empty[i % STAGES] : &full[i % STAGES], (i / STAGES) & 1u, wp, abort_flag, 2,
                   /*honour_abort=*/false);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    // the whole warp walks the tiles, one elected lane issues
    const bool issuer = elect_one();
    if (rank == 0) {
      uint32_t it = 0, tcount = 0, s = 0, ph = 0;
      bool ok = true;
      MxTile w;
      for (int tile = unit; ok && mx_tile<TR, FM>(p, offs, start, stile, tile, w); tile += units, ++tcount) {
        const uint32_t buf = tcount % DBUF;
        const uint32_t tph = (tcount / DBUF) & 1u;
        ok = wait_bounded(&tempty[buf], tph ^ 1u, wp, abort_flag, 3);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * TR;
        const uint32_t idesc = IDESC0 | (static_cast<uint32_t>(w.n >> 3) << 17);
        const bool all_scales = w.cols > 128 * (L::RA - 1);  // every scale tile along the rows is in use
        int kb = mx_first_k<PAIR>(w, p.k_blocks);
        for (int i_k = 0; i_k < p.k_blocks; ++i_k, ++it, kb = kb + 1 == p.k_blocks ? 0 : kb + 1) {
          ok = wait_bounded(&full[s], ph, wp, abort_flag, 4);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * L::A_BYTES);
          const uint32_t b0 = smem_u32(sB + s * L::B_BYTES);
          const uint32_t f0 = smem_u32(sSF + s * L::SF_BYTES);
          // scale columns of this stage: A's two tiles, then per k tile the rows' tiles side by side
          const uint32_t sfa = tmem_base + SF_COL + (it & 1u) * SF_SET;
          const uint32_t sfb = sfa + 8;
          const int steps = min(4, (p.K - kb * L::BK + 63) / 64);
          if (issuer) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (2 * h < steps) {
                copy_scales<PAIR>(sfa + h * 4, f0 + h * 512);
                copy_scales<PAIR>(sfb + h * (4 * L::RA), f0 + L::SF_TILE + h * 512);
                if (L::RA == 2 && all_scales)
                  copy_scales<PAIR>(sfb + h * (4 * L::RA) + 4, f0 + 2 * L::SF_TILE + h * 512);
              }
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < steps) {
                const uint32_t id = static_cast<uint32_t>(kk & 1) * 2u;  // which byte pair of the scale column
                umma_mxf4<PAIR>(d_tmem, smem_desc_sw128(a0 + kk * 32, 16, 1024), smem_desc_sw128(b0 + kk * 32, 16, 1024),
                                idesc | (id << 4) | (id << 29), sfa + (kk >> 1) * 4, sfb + (kk >> 1) * (4 * L::RA),
                                (i_k > 0 || kk > 0) ? 1u : 0u);
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
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int NCH = TR / 64;           // chunks of 32 rows a warp takes: one half of the tile's
    const uint32_t ew = warp & 3u;         // TMEM lane quarter
    const uint32_t eh = (warp - 2u) >> 2;  // half of the rows
    uint32_t tcount = 0;
    bool ok = true;
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(&tempty[0]), 0) : smem_u32(&tempty[0]);
    MxTile w;
    for (int tile = unit; mx_tile<TR, FM>(p, offs, start, stile, tile, w); tile += units, ++tcount) {
      const int fw = w.f0 + static_cast<int>(rank * 128u + ew * 32u);
      const int n = fw + static_cast<int>(lane);
      const int nvalid = max(0, min(32, p.N - fw));
      const uint32_t buf = tcount % DBUF;
      const uint32_t tph = (tcount / DBUF) & 1u;
      float bias_n = 0.f;
      if constexpr (AddsBias<EPI>::value)
        if (n < p.N) bias_n = load_bias<BF16>(p.bias, p.bias_f32, static_cast<int64_t>(w.e) * p.N + n);
      if (ok) ok = wait_bounded(&tfull[buf], tph, wp, abort_flag, 6);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;
      tc_fence_after();
      const uint32_t tbase = tmem_base + ((ew * 32u) << 16) + buf * TR;
      const int c_first = static_cast<int>(eh) * NCH;
      const auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_peer(tempty0 + buf * 8);
          else
            mbar_arrive(&tempty[buf]);
        }
      };
      const auto apply = [&](const uint32_t (&acc)[32], float (&v)[32]) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          v[j] = __uint_as_float(acc[j]) + bias_n;
          if constexpr (EPI == EPI_RELU_BIAS) v[j] = v[j] > 0.f ? v[j] : 0.f;
        }
        if constexpr (AppliesGelu<EPI>::value) gelu32(v);
      };
      const int64_t at0 = static_cast<int64_t>(w.c0) * p.N + fw;
      if constexpr (F32) {
        uint32_t acc[NCH][32];
#pragma unroll
        for (int i = 0; i < NCH; ++i)
          if ((c_first + i) * 32 < w.n) tmem_ld_32x32b_x32(tbase + (c_first + i) * 32, acc[i]);
        tmem_wait_ld();
        hand_back();
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int r0 = (c_first + i) * 32;
          if (r0 < w.cols) {
            float v[32];
            apply(acc[i], v);
            store_cols32(v, reinterpret_cast<float*>(p.out) + at0 + static_cast<int64_t>(r0) * p.N, p.N, w.cols - r0, nvalid);
          }
        }
      } else {
        // rounded and packed as they are read, two chunks at a time, so that a
        // tile takes 64 registers until it is stored
        uint32_t pk[NCH][16];
#pragma unroll
        for (int i = 0; i < NCH; i += 2) {
          uint32_t acc[2][32];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if ((c_first + i + h) * 32 < w.n) tmem_ld_32x32b_x32(tbase + (c_first + i + h) * 32, acc[h]);
          tmem_wait_ld();
          if (i + 2 == NCH) hand_back();
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if ((c_first + i + h) * 32 < w.n) {
              float v[32];
              apply(acc[h], v);
#pragma unroll
              for (int j = 0; j < 16; ++j) pk[i + h][j] = pack2<BF16>(v[2 * j], v[2 * j + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int r0 = (c_first + i) * 32;
          if (r0 < w.cols)
            store_packed16(pk[i], reinterpret_cast<uint16_t*>(p.out) + at0 + static_cast<int64_t>(r0) * p.N, p.N,
                           w.cols - r0, nvalid);
        }
      }
    }
  }

  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();  // neither CTA leaves while the other may still signal it
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace ge
