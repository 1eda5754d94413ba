// The mixture-of-experts layer with bf16 expert weights.
namespace qs {
namespace {
constexpr bool kFp4 = false;
}
}  // namespace qs

#include "moe_kernel.cuh"

namespace qs {
MoePlan plan_moe_bf16(int T, int d_model, int d_ff, int n_experts, int top_k, bool y_bf16) {
  return make_plan(T, d_model, d_ff, n_experts, top_k, y_bf16);
}
cudaError_t launch_moe_bf16(const MoeArgs& a, cudaStream_t s) { return launch(a, s); }
}  // namespace qs
