// The gated feed-forward layer in bf16 (see gated_product.hpp).
#include "gated_product.hpp"

namespace convmi {

hipError_t gated_fwd_bf16(const GatedArgs& a, hipStream_t s) { return gated_fwd<bf16_t>(a, s); }
hipError_t gated_bwd_bf16(const GatedArgs& a, hipStream_t s) { return gated_bwd<bf16_t>(a, s); }
GatedPlan gated_plan_bf16(int64_t rows, int C, int F) { return gated_plan<bf16_t>(rows, C, F); }
size_t gated_fwd_workspace_bf16(int64_t rows, int C, int F) { return gated_fwd_workspace<bf16_t>(rows, C, F); }

}  // namespace convmi
