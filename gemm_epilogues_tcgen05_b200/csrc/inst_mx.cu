// inst_mx.cu -- instances of the microscaled product.
#include "kernel_table.h"
#include "mx_kernel.cuh"

namespace ge_inst {

template <bool PAIR, int TR, int EPI, bool BF, bool F32>
MxInstance mx_one() {
  using L = ge::MxSmem<PAIR, TR>;
  return {ge::mx_kernel<PAIR, TR, EPI, BF, F32>, L::BYTES, 320, L::STAGES, L::BK};
}

template <bool PAIR, int TR, bool BF, bool F32>
MxInstance mx_epi(int epi) {
  switch (epi) {
    case ge::EPI_BIAS: return mx_one<PAIR, TR, ge::EPI_BIAS, BF, F32>();
    case ge::EPI_RELU_BIAS: return mx_one<PAIR, TR, ge::EPI_RELU_BIAS, BF, F32>();
    case ge::EPI_GELU_BIAS: return mx_one<PAIR, TR, ge::EPI_GELU_BIAS, BF, F32>();
    case ge::EPI_STORE: return mx_one<PAIR, TR, ge::EPI_STORE, BF, F32>();
    default: return {};
  }
}

template <bool PAIR, int TR>
MxInstance mx_tr(int epi, bool bf16, bool f32) {
  if (f32) return bf16 ? mx_epi<PAIR, TR, true, true>(epi) : mx_epi<PAIR, TR, false, true>(epi);
  return bf16 ? mx_epi<PAIR, TR, true, false>(epi) : mx_epi<PAIR, TR, false, false>(epi);
}

MxInstance mx_any(int tr, int epi, bool bf16, bool f32) {
  return tr == 256 ? mx_tr<true, 256>(epi, bf16, f32) : mx_tr<false, 128>(epi, bf16, f32);
}

}  // namespace ge_inst
