// inst_w4_f16.cu -- product with 4-bit weights, fp16 rows.
#include "inst_w4.cuh"

namespace ge_inst {
W4Instance w4_f16(int tp, bool gated, int ng) { return w4_any<false>(tp, gated, ng); }
}  // namespace ge_inst
