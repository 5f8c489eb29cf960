// gdn_lin_bf16.hip -- the linear-attention scan kernels for bf16 inputs.
#include "gdn_lin_scan.hpp"

namespace gdn {
hipError_t launch_lin_scan_bf16(const LinScan& A, LinMode mode, int64_t slots, hipStream_t stream) {
  switch (mode) {
    case kLinO: return lin_scan_mode<EngBF16, kLinO>(A, slots, stream);
    case kLinStF: return lin_scan_mode<EngBF16, kLinStF>(A, slots, stream);
    default: return lin_scan_mode<EngBF16, kLinDQ>(A, slots, stream);
  }
}
hipError_t launch_lin_sums_bf16(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream) {
  return lin_sums<EngBF16>(A, B, slots, stream);
}
hipError_t launch_lin_rev_bf16(const LinScan& A, const LinScan& B, int64_t slots, hipStream_t stream) {
  return lin_rev<EngBF16>(A, B, slots, stream);
}
}  // namespace gdn
