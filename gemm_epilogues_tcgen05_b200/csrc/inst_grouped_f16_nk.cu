// inst_grouped_f16_nk.cu -- expert-grouped kernels, fp16 operands, weights N x K.
#include "inst_grouped.cuh"

namespace ge_inst {
GroupedInstance grouped_f16_nk(int tr, int epi, bool split) { return grouped_any<false, true>(tr, epi, split); }
}  // namespace ge_inst
