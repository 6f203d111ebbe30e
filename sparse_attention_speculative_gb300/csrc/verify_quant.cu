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

// Whether every pair has a CTA of its own.  That takes up to t_max tiles one after the other
// instead of W / ctas, but no partial results, no kernel that merges them (together about
// 3 tiles' time), and, where many pairs share CTAs, no second part in a CTA (up to 5 more).
// With 12 tiles at most, since ranges follow the real lengths and this the longest.  Split and
// whole, us: one pair, 3 tiles 8.9 / 8.3, 5 tiles 8.9 / 10.1; 8 pairs, 2 tiles 11.4 / 9.1,
// 4 tiles 10.8 / 10.9, 6 tiles 11.0 / 13.0; 64 pairs of ragged single tokens, 6 tiles
// 15.1 / 10.7, 8 tiles 15.2 / 12.7; 128 pairs of 48 columns, 4 tiles 31.7 / 18.4, 8 tiles
// 41.0 / 25.8.
bool verify_quant_whole(const VerifyPlan& plan) {
  // (at most as many pairs as CTAs, of which a plan has no more than a CTA holds lengths)
  if (plan.pairs == 0 || plan.pairs > plan.ctas || plan.t_max > 12) return false;
  const int shared = plan.pairs * plan.t_max / plan.ctas;
  const int room = plan.pairs < 64 ? plan.pairs * 5 / 64 : 5;
  return plan.t_max - shared <= 3 + room;
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
