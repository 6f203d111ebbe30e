// verify_quant_d64.cu -- 8-bit-cache verification kernels instantiated for head_dim 64.
#include "verify_quant.cuh"

namespace vsd {
namespace verify_quant_detail {

cudaError_t launch_d64(const VerifyArgs& a, const QuantScales& s, const VerifyPlan& plan,
                        cudaStream_t stream) {
  return launch_quant_d<64>(a, s, plan, stream);
}

}  // namespace verify_quant_detail
}  // namespace vsd
