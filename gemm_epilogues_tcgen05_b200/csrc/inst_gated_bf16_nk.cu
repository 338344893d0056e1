// inst_gated_bf16_nk.cu -- gated layers, bf16 operands, N x K weight.
#include "inst_gated.cuh"

namespace ge_inst {
GatedInstance gated_bf16_nk(int bn, bool pair, int epi) { return gated_any<true, true>(bn, pair, epi); }
GatedSkinnyInstance gated_skinny_bf16_nk(int tp, int gn) { return gated_skinny_any<true, true>(tp, gn); }
}  // namespace ge_inst
