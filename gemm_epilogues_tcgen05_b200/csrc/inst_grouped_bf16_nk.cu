// inst_grouped_bf16_nk.cu -- expert-grouped kernels, bf16 operands, weights N x K.
#include "inst_grouped.cuh"

namespace ge_inst {
GroupedInstance grouped_bf16_nk(int tr, int epi, bool split) { return grouped_any<true, true>(tr, epi, split); }
}  // namespace ge_inst
