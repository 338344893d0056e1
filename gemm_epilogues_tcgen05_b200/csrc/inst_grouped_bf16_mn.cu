// inst_grouped_bf16_mn.cu -- expert-grouped kernels, bf16 operands, weights K x N.
#include "inst_grouped.cuh"

namespace ge_inst {
GroupedInstance grouped_bf16_mn(int tr, int epi, bool split) { return grouped_any<true, false>(tr, epi, split); }
}  // namespace ge_inst
