// inst_grouped.cuh -- instances of the expert-grouped kernel for one operand
// type and weight layout (included by inst_grouped_*.cu).
#pragma once

#include "grouped_kernel.cuh"
#include "kernel_table.h"

namespace ge_inst {

template <bool PAIR, int TR, int KPS, int EPI, bool BF, bool WK, bool SPLIT>
GroupedInstance grouped_one() {
  using L = ge::GroupedSmem<PAIR, TR, KPS>;
  return {ge::grouped_kernel<PAIR, TR, KPS, EPI, BF, WK, SPLIT>, L::BYTES, ge::GroupedThreads<EPI, TR>::value, L::STAGES,
          L::BK};
}

template <bool PAIR, int TR, int KPS, bool BF, bool WK, bool SPLIT>
GroupedInstance grouped_epi(int epi) {
  switch (epi) {
    case ge::EPI_BIAS: return grouped_one<PAIR, TR, KPS, ge::EPI_BIAS, BF, WK, SPLIT>();
    case ge::EPI_RELU_BIAS: return grouped_one<PAIR, TR, KPS, ge::EPI_RELU_BIAS, BF, WK, SPLIT>();
    case ge::EPI_RELU_AUX_BIAS: return grouped_one<PAIR, TR, KPS, ge::EPI_RELU_AUX_BIAS, BF, WK, SPLIT>();
    case ge::EPI_DRELU_BGRAD: return grouped_one<PAIR, TR, KPS, ge::EPI_DRELU_BGRAD, BF, WK, SPLIT>();
    case ge::EPI_GELU_BIAS: return grouped_one<PAIR, TR, KPS, ge::EPI_GELU_BIAS, BF, WK, SPLIT>();
    case ge::EPI_GELU_AUX_BIAS: return grouped_one<PAIR, TR, KPS, ge::EPI_GELU_AUX_BIAS, BF, WK, SPLIT>();
    case ge::EPI_STORE: return grouped_one<PAIR, TR, KPS, ge::EPI_STORE, BF, WK, SPLIT>();
    case ge::EPI_WGRAD:
      if constexpr (KPS == 1 && !WK) return grouped_one<PAIR, TR, KPS, ge::EPI_WGRAD, BF, WK, SPLIT>();
    default: return {};
  }
}

template <bool BF, bool WK>
GroupedInstance grouped_any(int tr, int epi, bool split) {
  if (tr == 32) return split ? grouped_epi<false, 32, 2, BF, WK, true>(epi) : grouped_epi<false, 32, 2, BF, WK, false>(epi);
  if (tr == 128) return split ? grouped_epi<false, 128, 1, BF, WK, true>(epi) : grouped_epi<false, 128, 1, BF, WK, false>(epi);
  if (tr == 256) return grouped_epi<true, 256, 1, BF, WK, false>(epi);
  return {};
}

}  // namespace ge_inst
