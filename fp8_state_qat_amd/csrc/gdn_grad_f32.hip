// gdn_grad_f32.hip -- the gradients of the gated delta rule for fp32 inputs.
#include "gdn_grad_kernels.hpp"

namespace gdn {

hipError_t launch_grad_f32(const gdn_shape_t& s, const GradArgs& a, int64_t items, hipStream_t stream) {
  return s.dk == 128 ? launch_grad<EngF32, 128>(s, a, items, stream) : launch_grad<EngF32, 64>(s, a, items, stream);
}

}  // namespace gdn
