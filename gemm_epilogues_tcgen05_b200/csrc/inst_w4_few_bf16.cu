// inst_w4_few_bf16.cu -- few bf16 rows times 4-bit weights, each warp alone.
#include "inst_w4_few.cuh"

namespace ge_inst {
W4FewInstance w4_few_bf16(int rows, bool gated, int ng) { return w4_few_any<true>(rows, gated, ng); }
}  // namespace ge_inst
