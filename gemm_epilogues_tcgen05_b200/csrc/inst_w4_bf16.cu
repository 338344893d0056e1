// inst_w4_bf16.cu -- product with 4-bit weights, bf16 rows.
#include "inst_w4.cuh"

namespace ge_inst {
W4Instance w4_bf16(int tp, bool gated, int ng) { return w4_any<true>(tp, gated, ng); }
}  // namespace ge_inst
