// inst_grouped_f16_mn.cu -- expert-grouped kernels, fp16 operands, weights K x N.
#include "inst_grouped.cuh"

namespace ge_inst {
GroupedInstance grouped_f16_mn(int tr, int epi, bool split) { return grouped_any<false, false>(tr, epi, split); }
}  // namespace ge_inst
