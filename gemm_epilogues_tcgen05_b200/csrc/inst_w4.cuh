// inst_w4.cuh -- kernel instances of the product with 4-bit weights for one type
// (included by inst_w4_*.cu).
#pragma once

#include "kernel_table.h"
#include "w4_kernel.cuh"

namespace ge_inst {

template <int TP, bool GATED, int NG, bool BF>
W4Instance w4_one() {
  using L = ge::W4Smem<TP, NG>;
  return {ge::w4_kernel<TP, GATED, NG, BF>, L::BYTES, L::THREADS, L::ACC, L::STAGES};
}

// tp at most 128 / ng (tensor memory), gated 64 (registers)
template <bool GATED, bool BF>
W4Instance w4_tp(int tp, int ng) {
  if (ng == 4) return tp == 16 ? w4_one<16, GATED, 4, BF>() : w4_one<32, GATED, 4, BF>();
  if (ng == 2)
    return tp == 16 ? w4_one<16, GATED, 2, BF>() : tp == 32 ? w4_one<32, GATED, 2, BF>() : w4_one<64, GATED, 2, BF>();
  if (tp == 16) return w4_one<16, GATED, 1, BF>();
  if (tp == 32) return w4_one<32, GATED, 1, BF>();
  if constexpr (!GATED)
    if (tp == 128) return w4_one<128, GATED, 1, BF>();
  return w4_one<64, GATED, 1, BF>();
}

template <bool BF>
W4Instance w4_any(int tp, bool gated, int ng) {
  return gated ? w4_tp<true, BF>(tp, ng) : w4_tp<false, BF>(tp, ng);
}

}  // namespace ge_inst
