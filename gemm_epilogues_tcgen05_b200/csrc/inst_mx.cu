// inst_mx.cu -- instances of the microscaled product.
#include "kernel_table.h"
#include "mx_kernel.cuh"

namespace ge_inst {

template <bool PAIR, int TR, int EPI, bool BF>
MxInstance mx_one() {
  using L = ge::MxSmem<PAIR, TR>;
  return {ge::mx_kernel<PAIR, TR, EPI, BF>, L::BYTES, 320, L::STAGES, L::BK};
}

template <bool PAIR, int TR, bool BF>
MxInstance mx_epi(int epi) {
  switch (epi) {
    case ge::EPI_BIAS: return mx_one<PAIR, TR, ge::EPI_BIAS, BF>();
    case ge::EPI_RELU_BIAS: return mx_one<PAIR, TR, ge::EPI_RELU_BIAS, BF>();
    case ge::EPI_GELU_BIAS: return mx_one<PAIR, TR, ge::EPI_GELU_BIAS, BF>();
    case ge::EPI_STORE: return mx_one<PAIR, TR, ge::EPI_STORE, BF>();
    default: return {};
  }
}

MxInstance mx_any(int tr, int epi, bool bf16) {
  if (tr == 256) return bf16 ? mx_epi<true, 256, true>(epi) : mx_epi<true, 256, false>(epi);
  return bf16 ? mx_epi<false, 128, true>(epi) : mx_epi<false, 128, false>(epi);
}

}  // namespace ge_inst
