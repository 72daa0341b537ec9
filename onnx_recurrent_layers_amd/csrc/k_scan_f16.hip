// k_scan_f16.hip -- the selective scan's kernels for f16 tensors (a file a type:
// they compile side by side).
#include "scan_grad_kernel.h"
#include "scan_kernel.h"

namespace rnnhip {

hipError_t launch_scan_local_f16(const ScanArgs& a, hipStream_t s) { return scan_of<f16_t, true>(a, s); }
hipError_t launch_scan_f16(const ScanArgs& a, hipStream_t s) { return scan_of<f16_t, false>(a, s); }
hipError_t launch_scan_backward_f16(const ScanArgs& a, hipStream_t s) { return scan_backward_of<f16_t>(a, s); }

}  // namespace rnnhip
