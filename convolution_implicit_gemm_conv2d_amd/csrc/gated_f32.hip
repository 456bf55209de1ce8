// The gated feed-forward layer in fp32 (see gated_product.hpp).
#include "gated_product.hpp"

namespace convmi {

hipError_t gated_fwd_f32(const GatedArgs& a, hipStream_t s) { return gated_fwd<float>(a, s); }
hipError_t gated_bwd_f32(const GatedArgs& a, hipStream_t s) { return gated_bwd<float>(a, s); }
GatedPlan gated_plan_f32(int64_t rows, int C, int F) { return gated_plan<float>(rows, C, F); }
size_t gated_fwd_workspace_f32(int64_t rows, int C, int F) { return gated_fwd_workspace<float>(rows, C, F); }

}  // namespace convmi
