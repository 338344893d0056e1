// inst_w4_few.cuh -- kernel instances of the product with 4-bit weights whose warps do
// all of it alone, for one type (included by inst_w4_few_*.cu).
#pragma once

#include "kernel_table.h"
#include "w4_few.cuh"

namespace ge_inst {

template <int NT, bool GATED, int NG, bool BF>
W4FewInstance w4_few_one() {
  return {{ge::w4_few_kernel<NT, GATED, NG, false, BF>, ge::w4_few_kernel<NT, GATED, NG, true, BF>},
          {ge::W4Few<NT, GATED ? 2 : 1, NG, false>::BYTES, ge::W4Few<NT, GATED ? 2 : 1, NG, true>::BYTES},
          32 * ge::kFewWarps, ge::W4Few<NT, GATED ? 2 : 1, NG, true>::DEPTH};
}

template <int NT, bool GATED, bool BF>
W4FewInstance w4_few_ng(int ng) {
  return ng == 1 ? w4_few_one<NT, GATED, 1, BF>() : ng == 2 ? w4_few_one<NT, GATED, 2, BF>() : w4_few_one<NT, GATED, 4, BF>();
}

template <bool BF>
W4FewInstance w4_few_any(int rows, bool gated, int ng) {
  if (rows <= 8) return gated ? w4_few_ng<1, true, BF>(ng) : w4_few_ng<1, false, BF>(ng);
  return gated ? w4_few_ng<2, true, BF>(ng) : w4_few_ng<2, false, BF>(ng);
}

}  // namespace ge_inst
