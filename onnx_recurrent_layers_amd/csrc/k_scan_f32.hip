// k_scan_f32.hip -- the selective scan's kernels for f32 tensors (a file a type:
// they compile side by side).
#include "scan_grad_kernel.h"
#include "scan_kernel.h"

namespace rnnhip {

hipError_t launch_scan_local_f32(const ScanArgs& a, hipStream_t s) { return scan_of<float, true>(a, s); }
hipError_t launch_scan_f32(const ScanArgs& a, hipStream_t s) { return scan_of<float, false>(a, s); }
hipError_t launch_scan_backward_f32(const ScanArgs& a, hipStream_t s) { return scan_backward_of<float>(a, s); }

}  // namespace rnnhip
