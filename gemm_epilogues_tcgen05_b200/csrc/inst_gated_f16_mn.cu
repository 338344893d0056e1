// inst_gated_f16_mn.cu -- gated layers, fp16 operands, K x N weight.
#include "inst_gated.cuh"

namespace ge_inst {
GatedInstance gated_f16_mn(int bn, bool pair, int epi) { return gated_any<false, false>(bn, pair, epi); }
GatedSkinnyInstance gated_skinny_f16_mn(int tp, int gn) { return gated_skinny_any<false, false>(tp, gn); }
}  // namespace ge_inst
