// inst_w4.cuh -- kernel instances of the product with 4-bit weights for one type
// (included by inst_w4_*.cu).
#pragma once

#include "kernel_table.h"
#include "w4_kernel.cuh"

namespace ge_inst {

template <int NT, bool GATED, int NG, bool BF>
W4Instance w4_one() {
  constexpr int MATS = GATED || NT >= 4 ? 2 : 1;
  using S = ge::W4Shape<NT>;
  return {ge::w4_kernel<NT, MATS, GATED, NG, BF>, S::WARPS, S::BUFS * S::WARPS * MATS * S::PART * 4};
}

template <int NT, bool BF>
W4Instance w4_nt(bool gated, int ng) {
  if (ng == 1) return gated ? w4_one<NT, true, 1, BF>() : w4_one<NT, false, 1, BF>();
  if (ng == 2) return gated ? w4_one<NT, true, 2, BF>() : w4_one<NT, false, 2, BF>();
  return gated ? w4_one<NT, true, 4, BF>() : w4_one<NT, false, 4, BF>();
}

template <bool BF>
W4Instance w4_any(int nt, bool gated, int ng) {
  return nt == 1   ? w4_nt<1, BF>(gated, ng)
         : nt == 2 ? w4_nt<2, BF>(gated, ng)
         : nt == 4 ? w4_nt<4, BF>(gated, ng)
                   : w4_nt<8, BF>(gated, ng);
}

}  // namespace ge_inst
