// inst_gated_bf16_mn.cu -- gated layers, bf16 operands, K x N weight.
#include "inst_gated.cuh"

namespace ge_inst {
GatedInstance gated_bf16_mn(int bn, bool pair, int epi) { return gated_any<true, false>(bn, pair, epi); }
GatedSkinnyInstance gated_skinny_bf16_mn(int tp, int gn) { return gated_skinny_any<true, false>(tp, gn); }
}  // namespace ge_inst
