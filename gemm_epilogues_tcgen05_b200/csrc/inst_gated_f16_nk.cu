// inst_gated_f16_nk.cu -- gated layers, fp16 operands, N x K weight.
#include "inst_gated.cuh"

namespace ge_inst {
GatedInstance gated_f16_nk(int bn, bool pair, int epi) { return gated_any<false, true>(bn, pair, epi); }
GatedSkinnyInstance gated_skinny_f16_nk(int tp, int gn) { return gated_skinny_any<false, true>(tp, gn); }
}  // namespace ge_inst
