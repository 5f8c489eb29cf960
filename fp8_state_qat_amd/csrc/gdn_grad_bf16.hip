// gdn_grad_bf16.hip -- the gradients of the gated delta rule for bf16 inputs.
#include "gdn_grad_kernels.hpp"

namespace gdn {

hipError_t launch_grad_bf16(const gdn_shape_t& s, const GradArgs& a, int64_t items, hipStream_t stream) {
  return s.dk == 128 ? launch_grad<EngBF16, 128>(s, a, items, stream) : launch_grad<EngBF16, 64>(s, a, items, stream);
}

}  // namespace gdn
