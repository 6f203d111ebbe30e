// verify_quant.cu -- host side of the 8-bit-cache verification: workspace size and the
// dispatch to the per-head-dimension instantiations (kernels in verify_quant.cuh; the grid
// is the bf16 call's, plan_verify; the kernel cuts the work up itself).
#include "launch.h"

namespace vsd {

namespace verify_quant_detail {
cudaError_t launch_d128(const VerifyArgs& a, const QuantScales& s, const VerifyPlan& plan,
                        cudaStream_t stream);
cudaError_t launch_d64(const VerifyArgs& a, const QuantScales& s, const VerifyPlan& plan,
                       cudaStream_t stream);
}  // namespace verify_quant_detail

size_t verify_quant_span_bytes(const VerifyPlan& plan) {
  return (static_cast<size_t>(plan.pairs) * 8 + 255) / 256 * 256;
}

size_t verify_quant_workspace_bytes(const VerifyPlan& plan, int head_dim) {
  if (plan.ctas <= 1 || plan.pairs == 0) return 0;
  return verify_quant_span_bytes(plan) +
         (static_cast<size_t>(plan.pairs) + plan.ctas) * plan.nq * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_verify_quant(const VerifyArgs& a, const QuantScales& s, const VerifyPlan& plan,
                                cudaStream_t stream) {
  if (plan.pairs == 0) return cudaSuccess;
  if (a.d == 128) return verify_quant_detail::launch_d128(a, s, plan, stream);
  if (a.d == 64) return verify_quant_detail::launch_d64(a, s, plan, stream);
  return cudaErrorInvalidValue;
}

}  // namespace vsd
