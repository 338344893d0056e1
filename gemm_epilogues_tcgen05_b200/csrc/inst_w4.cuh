// inst_w4.cuh -- kernel instances of the product with 4-bit weights for one type
// (included by inst_w4_*.cu).
#pragma once

#include "kernel_table.h"
#include "w4_kernel.cuh"

namespace ge_inst {

template <int TP, bool GATED, bool BF>
W4Instance w4_ng(int ng) {
  if (ng == 1) return {ge::w4_kernel<TP, GATED, 1, BF>, ge::W4Smem<TP, 1>::BYTES};
  if (ng == 2) return {ge::w4_kernel<TP, GATED, 2, BF>, ge::W4Smem<TP, 2>::BYTES};
  return {ge::w4_kernel<TP, GATED, 4, BF>, ge::W4Smem<TP, 4>::BYTES};
}

template <bool BF>
W4Instance w4_any(int tp, bool gated, int ng) {
  if (tp == 16) return gated ? w4_ng<16, true, BF>(ng) : w4_ng<16, false, BF>(ng);
  if (tp == 32) return gated ? w4_ng<32, true, BF>(ng) : w4_ng<32, false, BF>(ng);
  if (tp == 64) return gated ? w4_ng<64, true, BF>(ng) : w4_ng<64, false, BF>(ng);
  return gated ? W4Instance{} : w4_ng<128, false, BF>(ng);
}

}  // namespace ge_inst
