// w4_kernel.cuh -- rows times a weight held in 4 bits with group scales (layout:
// w4_quant.cuh), through tensor memory: Y[t][n] = epilog(sum_k X[t][k] s_g (q[n][k] - z_g)), and
// as a gated layer (two matrices). For many rows and large weights; what w4_few.cuh is
// for is measured at the plan.
//
// Swap-AB, as the few-row kernel: 128 features in the MMA's M slot, the rows of X,
// padded to TP, in its N slot. The weight's operand comes from tensor memory: a
// dequantising warp unpacks 32 columns of a lane's own feature to the integers q - z,
// exact in the 16-bit type (a shift, a mask with 128's or 1024's exponent, a subtraction
// for two), and stores them as 16 columns of its lane (tcgen05.st), so that
// no unpacked weight passes through shared memory. One MMA chain per group
// of G columns leaves the group's sums (fp32) in one of several accumulators, and
// accumulating warps add them, times the scale of their lane's feature, to sums in registers:
// no weight is rounded anywhere. K = 4096, N = 11008, G = 128: T = 64 22.7 us, T = 128 31.1,
// gated 39.4 and 58.2 (the codes alone 3.6 and 7.1 us); a product of the unpacked 16-bit weight reads
// 90 MB, 13.8 us, and the gated layer of it takes 35 us at T = 64.
//
// Warp roles:
//   first 16 or 8: dequantise: lane quarter warp % 4, every fourth (second) stage of
//           128 columns
//   then 8 or 16: accumulate and finish: lane quarter warp % 4, up to 32 rows, every
//           second stage (gated: the gate's, or the up projection's) but for TP = 128
//   then 1  X by TMA
//   last    tensor memory, MMAs
// What a stage costs is mostly the handing on between them, about 200 cycles a wait:
// with every role's work left out a stage took 500 ns when one set of accumulating
// warps took each of its groups' sums with a wait of its own.
// Codes, zeros and scales come in by cp.async, each warp its own, kW4Ahead blocks
// ahead of its work.
//
// Work split (stream-K): as the few-row kernel (skinny_kernel.cuh), blocks of 128
// columns instead of its k-blocks. A shared tile's parts are joined warp by warp, each
// with a ticket for its own lanes and rows: no accumulating warp waits for
// another, and the stages under way cover the ticket's round trip.
#pragma once

#include "activation.cuh"
#include "few_rows.cuh"
#include "skinny_kernel.cuh"
#include "w4_quant.cuh"

namespace ge {

struct W4MulParams {
  int32_t T, N, K;
  int32_t rt, kt;        // 32-feature tiles of a matrix, 128-column blocks
  int32_t total;         // 128-feature tiles x kt
  int32_t max_segs;
  int32_t epi, act;      // EpiKind; gated: an ActKind
  int32_t bias_f32, out_f32;
  FewSplit few;          // w4_few_kernel alone, and X
  const void* X;
  const uint8_t* q;
  const void* scales;
  const uint8_t* zeros;
  const void* bias;
  void* out;
  float* partials;       // [row blocks][tiles][max_segs][matrices][TP][128]
  int* tickets;          // [row blocks][tiles][accumulating warps], zero between launches
  int* status;
  uint64_t timeout_ns;
  int32_t inject_stall;
};

constexpr int kW4Ahead = 3;    // blocks that a warp's copies run ahead

template <int TP, int NG>
struct W4Smem {
  // A stage is 128 columns: the unpacked weights (64 columns of tensor memory), X, and an
  // accumulator for each group: as many stages as fit, an even number.
  static constexpr int STAGES = 6 * (64 + NG * TP) <= 512 ? 6 : 4 * (64 + NG * TP) <= 512 ? 4 : 2;
  static constexpr uint32_t X_SUB = TP * kBK * 2;             // TP rows x 64 columns
  static constexpr uint32_t X_BYTES = 2 * X_SUB;
  static constexpr int ROWS = TP < 32 ? TP : 32;              // of an accumulating warp
  static constexpr int PARTS = TP / ROWS, SETS = TP <= 64 ? 2 : 1;
  static constexpr int ACC = 4 * PARTS * SETS;                // accumulating warps
  // dequantising warps: at most one set of four a stage, or a set would wait for a
  // barrier two phases ahead and take it for this one
  static constexpr int DQ = ACC == 8 && STAGES >= 4 ? 16 : 8;
  static constexpr int THREADS = 32 * (DQ + ACC + 2);
  static constexpr uint32_t CODES = 2048 + 32 * NG;           // of a dequantising warp and block: codes, zeros
  static constexpr uint32_t SCALES = 64 * NG;                 // of an accumulating warp and block
  static constexpr uint32_t OFF_X = 0;
  static constexpr uint32_t OFF_CODES = OFF_X + STAGES * X_BYTES;
  static constexpr uint32_t OFF_SCALES = OFF_CODES + DQ * kW4Ahead * CODES;
  static constexpr uint32_t OFF_JOIN = OFF_SCALES + ACC * kW4Ahead * SCALES;  // the second set's sums: [TP][128]
  static constexpr uint32_t OFF_BAR = OFF_JOIN + (SETS == 2 ? TP * 128 * 4 : 0);
  static constexpr uint32_t N_BARS = 4 * STAGES + 1;
  static constexpr uint32_t OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr uint32_t BYTES = OFF_MISC + 16 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_A = 0, COL_D = STAGES * 64;
  static_assert(COL_D + STAGES * NG * TP <= TMEM_COLS, "tensor memory columns");
  static_assert(BYTES <= 232448, "above the per-CTA limit");
  static_assert(DQ / 4 <= STAGES, "a set of dequantising warps a stage at most");
};

__device__ __forceinline__ void w4_copy_16(uint32_t saddr, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(saddr), "l"(src), "l"(policy) : "memory");
}

// one test of two phases, the second's while the first's is under way (either takes
// about 200 cycles, and a stage's products little more)
__device__ __forceinline__ bool mbar_try_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4, 20000;\n\t"
      "and.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb)
      : "memory");
  return done != 0;
}

template <bool BF16>
__device__ __forceinline__ uint32_t w4_sub(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// (a & b) | c in one instruction (of the expression the compiler makes two)
__device__ __forceinline__ uint32_t w4_and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The eight codes of a word less their zero point z (0 .. 127), as four operand
// registers. bf16: 128 + q - (128 + z), the codes below 128's exponent. fp16 has room
// for a nibble and the next: 1024 + q - (1024 + z), and (1024 + 16 q) / 16 - (64 + z) of the
// one above, which saves two of three shifts (they, and the logical operations, run at
// half rate: unpacking is what bounds a block).
template <bool BF16>
struct W4Unpack {
  uint32_t zero, zero16;
  __device__ __forceinline__ explicit W4Unpack(uint32_t z) {
    zero = z * 0x00010001u + (BF16 ? 0x43004300u : 0x64006400u);  // (one multiply-add: z is below 128)
    const __half2 n = __hneg2(__hsub2(*reinterpret_cast<const __half2*>(&zero), __float2half2_rn(960.f)));  // -(64 + z)
    zero16 = BF16 ? 0u : *reinterpret_cast<const uint32_t*>(&n);
  }
  template <int R>
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&r)[R], int at) const {
    if constexpr (BF16) {
#pragma unroll
      for (int m = 0; m < 4; ++m) r[at + m] = w4_sub<true>(w4_and_or(w >> (4 * m), 0x000f000fu, 0x43004300u), zero);
    } else {
#pragma unroll
      for (int m = 0; m < 4; m += 2) {
        const uint32_t v = w >> (4 * m);
        r[at + m] = w4_sub<false>(w4_and_or(v, 0x000f000fu, 0x64006400u), zero);
        const uint32_t hi = w4_and_or(v, 0x00f000f0u, 0x64006400u);
        const __half2 f = __hfma2(*reinterpret_cast<const __half2*>(&hi), __float2half2_rn(0.0625f),
                                  *reinterpret_cast<const __half2*>(&zero16));
        r[at + m + 1] = *reinterpret_cast<const uint32_t*>(&f);
      }
    }
  }
};

// 16 registers to 16 columns of this warp's lane quarter
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]: A's 16 k of a row are 8 columns of its lane
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One output from its sums (gated: gate and up projection), feature n of row t.
template <bool GATED, bool BF16>
__device__ __forceinline__ void w4_output(const W4MulParams& p, float a, float b, int t, int n, float bias_a, float bias_b) {
  a += bias_a;
  if (GATED || p.epi == EPI_GELU_BIAS) {
    float z[2] = {a, a}, v[2], none[2];
    act_values<2, false>(GATED ? p.act : ACT_GELU, z, v, none);
    a = GATED ? v[0] * (b + bias_b) : v[0];
  } else if (p.epi == EPI_RELU_BIAS) {
    a = a > 0.f ? a : 0.f;
  }
  const int64_t o = static_cast<int64_t>(t) * p.N + n;
  if (p.out_f32)
    reinterpret_cast<float*>(p.out)[o] = a;
  else
    reinterpret_cast<uint16_t*>(p.out)[o] = w4_round16<BF16>(a);
}

template <int TP, bool GATED, int NG, bool BF16>
__global__ void __launch_bounds__(W4Smem<TP, NG>::THREADS, 1)
    w4_kernel(const __grid_constant__ CUtensorMap tmX, const W4MulParams p) {
  using L = W4Smem<TP, NG>;
  constexpr int MATS = GATED ? 2 : 1, STAGES = L::STAGES, AHEAD = kW4Ahead;
  constexpr int XS = STAGES / MATS;  // stages of X: both matrices' share one
  constexpr int DQ = L::DQ, ACC = L::ACC, ROWS = L::ROWS;
  static_assert(MATS == 1 || L::SETS == 2, "a gated layer's matrices have a set of accumulating warps each");
  constexpr uint32_t IDESC = idesc_f16(BF16, false, false, 128, TP);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // afull   the dequantising warps of a stage have stored (4 arrivals)
  // xfull   X has come (transaction bytes)
  // dfull   a stage's products are complete (commit)
  // sfree   the accumulating warps have read a stage's sums: everything of the stage,
  //         the unpacked weights and X that its products read, may be replaced
  uint64_t* afull = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* xfull = afull + STAGES;
  uint64_t* sfree = xfull + STAGES;
  uint64_t* dfull = sfree + STAGES;
  uint64_t* drain = dfull + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

  const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
  const int row0 = blockIdx.y * TP;
  SkinnyParams sp{};  // what a segment is found by
  sp.kbt = p.kt;
  sp.total_kb = p.total;
  const uint32_t lo = static_cast<uint32_t>(static_cast<uint64_t>(blockIdx.x) * p.total / gridDim.x);
  const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(blockIdx.x + 1) * p.total / gridDim.x);
  TileParams wp{};
  wp.status = p.status;
  wp.timeout_ns = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&afull[s], 4);
      mbar_init(&xfull[s], 1);
      mbar_init(&sfree[s], 4 * L::PARTS);
      mbar_init(&dfull[s], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == DQ + ACC && lane == 0) prefetch_tensormap(&tmX);
  if (warp == DQ + ACC + 1) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  wait_for_inputs();

  // blocks lo .. hi - 1 of (tile, kb), the matrices of each one after the other
  if (warp < DQ) {
    // --------------------------------------------------------- dequantise
    // steps set, set + SETS, ... of (hi - lo) MATS
    constexpr uint32_t SETS = DQ / 4, KB_STEP = SETS / MATS;
    const uint32_t quarter = warp & 3u, set = warp >> 2;
    const uint32_t ring = smem_u32(smem + L::OFF_CODES) + warp * (AHEAD * L::CODES), end = ring + AHEAD * L::CODES;
    const uint64_t policy = l2_policy_evict_first();
    const uint32_t kt = static_cast<uint32_t>(p.kt), steps = (hi - lo) * MATS;
    const bool zeros = p.zeros != nullptr;
    uint32_t i_in = 4 * (lo / kt) + quarter, kb_in = lo % kt + set / MATS, step_in = set, place_in = ring;
    int64_t tile = (static_cast<int64_t>(set % MATS) * p.rt + i_in) * p.kt + kb_in;
    const auto settle = [&]() {
      while (kb_in >= kt) {
        kb_in -= kt;
        i_in += 4;
        tile += 3 * static_cast<int64_t>(kt);
      }
    };
    settle();
    const auto fetch = [&]() {
      if (step_in < steps) {
        if (i_in < static_cast<uint32_t>(p.rt)) {
          const uint8_t* q = p.q + tile * kW4TileBytes + lane * 16;
#pragma unroll
          for (int b = 0; b < 4; ++b) w4_copy_16(place_in + 512 * b + lane * 16, q + 512 * b, policy);
          if (zeros && lane < 2 * NG) w4_copy_16(place_in + 2048 + lane * 16, p.zeros + tile * (32 * NG) + lane * 16, policy);
        }
        kb_in += KB_STEP;
        tile += KB_STEP;
        settle();
        place_in = place_in + L::CODES == end ? ring : place_in + L::CODES;
        step_in += SETS;
      }
      cp_async_commit();
    };
    for (int d = 0; d < AHEAD; ++d) fetch();
    uint32_t place = ring;
    bool ok = true;
    for (uint32_t it = set; it < steps; it += SETS) {
      const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
      cp_async_wait<AHEAD - 1>();
      if (zeros) __syncwarp();  // (codes are copied and read by one lane)
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(&sfree[s], ph ^ 1u, wp, abort_flag, 1));
      if (ok) {
        tc_fence_after();
        const uint32_t a = tmem_base + ((quarter * 32u) << 16) + L::COL_A + s * 64;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint4 c = ld_shared_v4(place + 512 * b + lane * 16);
          const W4Unpack<BF16> unpack(zeros ? ld_shared_u8(place + 2048 + b * NG / 4 * 32 + lane) : 8u);
          uint32_t r[16];
          unpack(c.x, r, 0);
          unpack(c.y, r, 4);
          unpack(c.z, r, 8);
          unpack(c.w, r, 12);
          tmem_st_32x32b_x16(a + 16 * b, r);
        }
      }
      if (zeros) __syncwarp();
      fetch();
      place = place + L::CODES == end ? ring : place + L::CODES;
      if (!ok) continue;  // (the copies under way are waited for below)
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&afull[s]);
    }
    cp_async_wait<0>();
  } else if (warp < DQ + ACC) {
    // ------------------------------------------- accumulate, join, finish
    const uint32_t aw = warp - DQ, quarter = warp & 3u, part = (aw >> 2) % L::PARTS;  // part: rows ROWS part .. of TP
    const uint32_t set = (aw >> 2) / L::PARTS;                                        // steps set, set + SETS, ...
    constexpr uint32_t SETS = L::SETS, KB_STEP = SETS / MATS;
    const uint32_t ring = smem_u32(smem + L::OFF_SCALES) + aw * (AHEAD * L::SCALES), end = ring + AHEAD * L::SCALES;
    float* join = reinterpret_cast<float*>(smem + L::OFF_JOIN) + part * (ROWS * 128) + quarter * 32 + lane;
    const uint32_t join_bar = 1 + part * 4 + quarter;
    const uint64_t policy = l2_policy_evict_first();
    const uint32_t kt = static_cast<uint32_t>(p.kt), steps = (hi - lo) * MATS;
    uint32_t i_in = 4 * (lo / kt) + quarter, kb_in = lo % kt + set / MATS, step_in = set, place_in = ring;
    int64_t tile = (static_cast<int64_t>(set % MATS) * p.rt + i_in) * p.kt + kb_in;
    const auto settle = [&]() {
      while (kb_in >= kt) {
        kb_in -= kt;
        i_in += 4;
        tile += 3 * static_cast<int64_t>(kt);
      }
    };
    settle();
    const auto fetch = [&]() {
      if (step_in < steps) {
        if (i_in < static_cast<uint32_t>(p.rt) && lane < 4 * NG)
          w4_copy_16(place_in + lane * 16, reinterpret_cast<const uint8_t*>(p.scales) + tile * (64 * NG) + lane * 16, policy);
        kb_in += KB_STEP;
        tile += KB_STEP;
        settle();
        place_in = place_in + L::SCALES == end ? ring : place_in + L::SCALES;
        step_in += SETS;
      }
      cp_async_commit();
    };
    for (int d = 0; d < AHEAD; ++d) fetch();
    uint32_t place = ring, it = set, seg_end = 0;
    bool ok = true;
    uint32_t gpos = lo;
    Segment seg;
    while (skinny_segment(sp, hi, gpos, seg)) {
      const int n_local = static_cast<int>(quarter * 32 + lane), n = seg.tile * 128 + n_local;
      const bool n_ok = n < p.N;
      seg_end += static_cast<uint32_t>(seg.kb1 - seg.kb0) * MATS;
      float acc[ROWS];
#pragma unroll
      for (int t = 0; t < ROWS; ++t) acc[t] = 0.f;
      for (; it < seg_end; it += SETS) {
        const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
        cp_async_wait<AHEAD - 1>();
        __syncwarp();
        float sc[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k)
          sc[k] = w4_float<BF16>(static_cast<uint16_t>(ld_shared_u16(place + k * 64 + lane * 2)));
        if (ok) ok = __all_sync(0xffffffffu, wait_bounded(&dfull[s], ph, wp, abort_flag, 6));
        if (ok) {
          tc_fence_after();
          const uint32_t d = tmem_base + ((quarter * 32u) << 16) + L::COL_D + s * (NG * TP) + part * ROWS;
          constexpr int G2 = ROWS == 16 && NG > 1 ? 2 : 1;  // groups whose loads are in flight
#pragma unroll
          for (int k = 0; k < NG; k += G2) {
#pragma unroll
            for (int t0 = 0; t0 < ROWS; t0 += 16) {
              uint32_t r[G2][16];
#pragma unroll
              for (int e = 0; e < G2; ++e) tmem_ld_32x32b_x16(d + (k + e) * TP + t0, r[e]);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < G2; ++e)
#pragma unroll
                for (int t = 0; t < 16; ++t) acc[t0 + t] = fmaf(sc[k + e], __uint_as_float(r[e][t]), acc[t0 + t]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfree[s]);
        }
        __syncwarp();
        fetch();
        place = place + L::SCALES == end ? ring : place + L::SCALES;
      }
      // the second set's sums to the first: the other half of the columns', or the up projection's
      float up[MATS == 2 ? ROWS : 1];
      if constexpr (SETS == 2) {
        if (set == 1) {
#pragma unroll
          for (int t = 0; t < ROWS; ++t) join[t * 128] = acc[t];
          named_bar_sync(join_bar, 64);
          named_bar_sync(join_bar, 64);  // it has been read
          continue;
        }
        named_bar_sync(join_bar, 64);
#pragma unroll
        for (int t = 0; t < ROWS; ++t) {
          if constexpr (MATS == 2)
            up[t] = join[t * 128];
          else
            acc[t] += join[t * 128];
        }
        named_bar_sync(join_bar, 64);
      }
      const bool whole = seg.kb0 == 0 && seg.kb1 == p.kt;
      float bias_a = 0.f, bias_b = 0.f;
      if (p.bias && n_ok) {
        bias_a = load_bias<BF16>(p.bias, p.bias_f32, n);
        if constexpr (GATED) bias_b = load_bias<BF16>(p.bias, p.bias_f32, p.N + n);
      }
      const int t0 = static_cast<int>(part) * ROWS;
      if (whole) {
#pragma unroll
        for (int t = 0; t < ROWS; ++t)
          if (ok && n_ok && row0 + t0 + t < p.T)
            w4_output<GATED, BF16>(p, acc[t], MATS == 2 ? up[MATS == 2 ? t : 0] : 0.f, row0 + t0 + t, n, bias_a, bias_b);
        continue;
      }
      // this segment's sums, a ticket; the last segment's warp finishes its lanes and rows
      const int64_t tiles = p.total / p.kt, at = blockIdx.y * tiles + seg.tile;
      constexpr int64_t SEG = MATS * TP * 128;
      float* slots = p.partials + at * p.max_segs * SEG + t0 * 128 + n_local;
      float* own = slots + seg.seg * SEG;
#pragma unroll
      for (int t = 0; t < ROWS; ++t)
        if (row0 + t0 + t < p.T) {
          own[t * 128] = acc[t];
          if constexpr (MATS == 2) own[(TP + t) * 128] = up[t];
        }
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0 && ok) {
        int* ticket = p.tickets + at * ACC + aw;  // (of the first set's warps)
        last = atomicAdd(ticket, 1) == seg.nsegs - 1;
        if (last) *ticket = 0;  // ready for the next launch
      }
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __threadfence();
      constexpr int B = MATS == 2 ? 4 : 8;  // rows whose loads of (four / MATS) segments are in flight
#pragma unroll 1
      for (int b = 0; b < ROWS; b += B) {
        if (row0 + t0 + b >= p.T) break;
        float sum[MATS][B];
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
          for (int t = 0; t < B; ++t) sum[m][t] = 0.f;
        for (int s0 = 0; s0 < seg.nsegs; s0 += 4 / MATS) {
          float x[4 / MATS][MATS][B];
#pragma unroll
          for (int k = 0; k < 4 / MATS; ++k)
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
              for (int t = 0; t < B; ++t)
                x[k][m][t] = s0 + k < seg.nsegs && row0 + t0 + b + t < p.T
                                 ? __ldcg(slots + (s0 + k) * SEG + (m * TP + b + t) * 128)
                                 : 0.f;
#pragma unroll
          for (int k = 0; k < 4 / MATS; ++k)
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
              for (int t = 0; t < B; ++t) sum[m][t] += x[k][m][t];
        }
#pragma unroll
        for (int t = 0; t < B; ++t)
          if (n_ok && row0 + t0 + b + t < p.T)
            w4_output<GATED, BF16>(p, sum[0][t], sum[MATS - 1][t], row0 + t0 + b + t, n, bias_a, bias_b);
      }
    }
    cp_async_wait<0>();
  } else if (warp == DQ + ACC) {
    // ------------------------------------------------------------------- X
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_last();
      uint32_t it = 0, kb = lo % static_cast<uint32_t>(p.kt);
      for (uint32_t b = lo; b < hi; ++b, ++it) {
        // (a place is free when the last of the stages that read it is)
        const uint32_t s = it % XS, last = it * MATS + MATS - 1;
        if (!wait_bounded(&sfree[last % STAGES], ((last / STAGES) & 1u) ^ 1u, wp, abort_flag, 2)) break;
        mbar_arrive_expect_tx(&xfull[s], L::X_BYTES);
        uint8_t* x = smem + L::OFF_X + s * L::X_BYTES;
        const int k = static_cast<int>(kb) * 128;
        tma_load_2d_hint(x, &tmX, &xfull[s], k, row0, policy);
        tma_load_2d_hint(x + L::X_SUB, &tmX, &xfull[s], k + 64, row0, policy);
        if (++kb == static_cast<uint32_t>(p.kt)) kb = 0;
      }
      // what was issued lands before the CTA leaves
      const uint32_t inflight = it < XS ? it : XS;
      for (uint32_t i = it - inflight; i < it; ++i)
        wait_bounded(&xfull[i % XS], (i / XS) & 1u, wp, abort_flag, 3, /*honour_abort=*/false);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------------- MMA
    const bool issuer = elect_one();
    const uint32_t steps = (hi - lo) * MATS;
    for (uint32_t it = 0; it < steps; ++it) {
      const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u, xi = it / MATS, xs = xi % XS, xph = (xi / XS) & 1u;
      bool ok = mbar_try_wait2(&afull[s], ph, &xfull[xs], xph);
      if (!ok) ok = wait_bounded(&xfull[xs], xph, wp, abort_flag, 4) && wait_bounded(&afull[s], ph, wp, abort_flag, 5);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (issuer) {
        const uint32_t x = smem_u32(smem + L::OFF_X + xs * L::X_BYTES);
        const uint32_t a = tmem_base + L::COL_A + s * 64, d = tmem_base + L::COL_D + s * (NG * TP);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {  // 16 columns each
          constexpr int PER = 8 / NG;     // of them in a group
          const uint64_t bdesc = smem_desc_sw128(x + (kk >> 2) * L::X_SUB + (kk & 3) * 32, 16, 1024);
          umma_f16_ts(d + kk / PER * TP, a + kk * 8, bdesc, IDESC, kk % PER > 0 ? 1u : 0u);
          // (fault injection: the accumulating warps then wait for sums that are never announced)
          if (kk == 7 && !(p.inject_stall && it == 0 && (p.inject_stall == 1 || (blockIdx.x | blockIdx.y) == 0))) umma_commit(&dfull[s]);
        }
      }
    }
    if (issuer) umma_commit(drain);
    wait_bounded(drain, 0, wp, abort_flag, 8, /*honour_abort=*/false);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == DQ + ACC + 1) tmem_dealloc(tmem_base, L::TMEM_COLS);
}

}  // namespace ge
