// inst_gated_few.cu -- gated layers of at most 16 rows, each warp alone.
#include "gated_few.cuh"
#include "kernel_table.h"

namespace ge_inst {
namespace {
template <int NT, bool NK, bool BF>
GatedFewInstance one() {
  return {ge::gated_few_kernel<NT, NK, BF>, ge::GatedFew<NT>::BYTES};
}
template <int NT>
GatedFewInstance any(bool bf16, bool w_nk) {
  if (bf16) return w_nk ? one<NT, true, true>() : one<NT, false, true>();
  return w_nk ? one<NT, true, false>() : one<NT, false, false>();
}
}  // namespace
GatedFewInstance gated_few(bool bf16, bool w_nk, int rows) { return rows <= 8 ? any<1>(bf16, w_nk) : any<2>(bf16, w_nk); }
}  // namespace ge_inst
