// gdn_lin_f32.hip -- the linear-attention scan kernels for fp32 inputs.
#include "gdn_lin_scan.hpp"

namespace gdn {
hipError_t launch_lin_scan_f32(const LinScan& A, LinMode mode, int64_t slots, hipStream_t stream) {
  switch (mode) {
    case kLinO: return lin_scan_mode<EngF32, kLinO>(A, slots, stream);
    case kLinStF: return lin_scan_mode<EngF32, kLinStF>(A, slots, stream);
    default: return lin_scan_mode<EngF32, kLinDQ>(A, slots, stream);
  }
}
hipError_t launch_lin_sums_f32(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream) {
  return lin_sums<EngF32>(A, B, slots, stream);
}
hipError_t launch_lin_rev_f32(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream) {
  return lin_rev<EngF32>(A, B, slots, stream);
}
}  // namespace gdn
