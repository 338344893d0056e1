// few_rows.cuh -- what the kernels of few rows share whose warps work alone (w4_few.cuh,
// gated_few.cuh): the split of a weight's tiles of 32 features among clusters, CTAs and
// warps, the product of fragments, and the join of the warps' sums.
#pragma once

#include "ptx.cuh"

namespace ge {

constexpr int kFewWarps = 16;
constexpr int kFewLd = 36;  // floats between the rows of kept sums: no two lanes in a bank

// log2 of the CTAs of a cluster; what a cluster has of the half rows of tiles, and its CTAs
// of the columns of tiles (the first `rest` one more)
struct FewSplit {
  int32_t split;
  uint32_t half_quot, half_rest, kt_quot, kt_rest;
};

template <bool BF16>
__device__ __forceinline__ void few_mma(float (&d)[4], bool zero, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
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

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// The tiles of a CTA's half rows [h0, h1) of tiles, nkb columns of tiles wide, row after row.
// A tile that both halves are wanted of weighs 2, one of the first or last row
// may weigh 1; the warps have equal shares of the weight, runs of tiles. (No divisions:
// a handful of them ahead of the first load, and in the join, cost 3 us.)
template <int H>
struct FewHalf {
  static constexpr int value = H;
};

struct FewRuns {
  uint32_t nkb, row0, rows, first, last_at, weight;  // rows of tiles; first: log2 of the weight of the first row's tiles
  __device__ __forceinline__ FewRuns(uint32_t h0, uint32_t h1, uint32_t nkb_) : nkb(nkb_), row0(h0 >> 1) {
    rows = ((h1 + 1) >> 1) - row0;
    first = (h0 & 1u) || h1 - h0 == 1 ? 0 : 1;
    weight = (h1 - h0) * nkb;
    last_at = (h1 & 1u) && rows > 1 ? weight - nkb : weight;  // weight ahead of a last row that weighs 1
  }
  // the first tile of warp w: of the tiles that begin at its share or later
  __device__ __forceinline__ uint32_t begin(uint32_t w) const {
    const uint32_t x = weight * w / kFewWarps;
    if (x <= nkb << first) return (x + first) >> first;
    if (x <= last_at) return nkb + ((x - (nkb << first) + 1) >> 1);
    return (rows - 1) * nkb + x - last_at;
  }
};

// one of `parts` shares of `total` = quot parts + rest
__device__ __forceinline__ uint32_t few_share(uint32_t i, uint32_t quot, uint32_t rest) { return i * quot + min(i, rest); }

// The sums that warps have kept, added in a fixed order and handed to out(row of tiles, row of
// X, sum, second matrix's sum), a lane its feature. A warp's first row of tiles is RING
// bytes into its WARP, its last one at the start: [matrix][8 NT rows of X][kFewLd]; behind the warps'
// memory, `kept`: the row of tiles of each (first, last), -1 for none. A warp takes a row of
// X (of a cluster's, the CTAs in turn).
template <int NT, int MATS, uint32_t WARP, uint32_t RING, class Out>
__device__ __forceinline__ void few_join(uint8_t* smem, int log_split, uint32_t rank, int T, const Out& out) {
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  __syncwarp();
  if (log_split)
    cluster_sync();
  else
    __syncthreads();
  // lane e holds entry e
  const int own = reinterpret_cast<const int*>(smem + kFewWarps * WARP)[lane];
  const uint32_t same = __match_any_sync(0xffffffffu, own);
  uint32_t leaders = __ballot_sync(0xffffffffu, own >= 0 && (same & ((1u << lane) - 1u)) == 0);
  uint32_t t = rank * kFewWarps + warp;
  for (; leaders; leaders &= leaders - 1) {
    const int r = __shfl_sync(0xffffffffu, own, __ffs(leaders) - 1);
    for (; t < static_cast<uint32_t>(T); t += kFewWarps << log_split) {
      float a = 0.f, b = 0.f;
      for (uint32_t s = 0; s < 1u << log_split; ++s) {
        const uint32_t base = log_split ? mapa_shared(smem_u32(smem), s) : smem_u32(smem);
        uint32_t from = __ballot_sync(0xffffffffu, static_cast<int>(ld_cluster_u32(base + kFewWarps * WARP + 4 * lane)) == r);
        for (; from; from &= from - 1) {
          const uint32_t e = __ffs(from) - 1;
          const uint32_t at = base + (e >> 1) * WARP + (e & 1u ? 0 : RING) + (t * kFewLd + lane) * 4;
          a += __uint_as_float(ld_cluster_u32(at));
          if constexpr (MATS == 2) b += __uint_as_float(ld_cluster_u32(at + NT * 8 * kFewLd * 4));
        }
      }
      out(static_cast<uint32_t>(r), t, a, b);
    }
    t -= static_cast<uint32_t>(T);
  }
  __syncwarp();
  if (log_split) cluster_sync();  // (sums that another CTA reads)
}

}  // namespace ge
