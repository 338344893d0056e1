// inst_gated.cuh -- kernel instances of gated layers for one operand type and
// weight layout (included by inst_gated_*.cu).
#pragma once

#include "kernel_table.h"
#include "skinny_kernel.cuh"
#include "tile2_kernel.cuh"

namespace ge_inst {

template <int BN, int ST, int EPI, bool BF, bool BK>
GatedInstance gated_tile() {
  static_assert(ge::TileSmem<BN, ST, EPI>::BYTES <= 232448, "above the per-CTA limit");
  return {ge::tile_kernel<BN, ST, EPI, BF, BK>, ge::TileSmem<BN, ST, EPI>::BYTES, ge::kThreads, ST};
}

template <int ST, int EPI, bool BF, bool BK>
GatedInstance gated_pair() {
  using L = ge::Tile2Smem<256, ST, 8, EPI>;
  static_assert(L::BYTES <= 232448, "above the per-CTA limit");
  return {ge::tile2_kernel<256, ST, EPI, BF, BK>, L::BYTES, 64 + 32 * 8, ST};
}

template <bool BF, bool BK>
GatedInstance gated_any(int bn, bool pair, int epi) {
  constexpr int F = ge::EPI_GATED, B = ge::EPI_DGATED;
  if (pair) return epi == F ? gated_pair<5, F, BF, BK>() : gated_pair<5, B, BF, BK>();
  if (bn == 256) return epi == F ? gated_tile<256, 4, F, BF, BK>() : gated_tile<256, 4, B, BF, BK>();
  if (bn == 128) return epi == F ? gated_tile<128, 6, F, BF, BK>() : gated_tile<128, 6, B, BF, BK>();
  if (bn == 64 && epi == B) return gated_tile<64, 8, B, BF, BK>();
  return {};
}

template <int TP, int GN, bool BF, bool BK>
GatedSkinnyInstance gated_skinny_tp() {
  using L = ge::SkinnySmem<TP, 2, GN>;
  return {ge::skinny_kernel<TP, 2, ge::EPI_GATED, BF, BK, GN>, L::BYTES, L::STAGES};
}

template <bool BF, bool BK>
GatedSkinnyInstance gated_skinny_any(int tp, int gn) {
  if (tp == 16) return gn == 128 ? gated_skinny_tp<16, 128, BF, BK>() : gated_skinny_tp<16, 64, BF, BK>();
  return gn == 128 ? gated_skinny_tp<32, 128, BF, BK>() : gated_skinny_tp<32, 64, BF, BK>();
}

}  // namespace ge_inst
