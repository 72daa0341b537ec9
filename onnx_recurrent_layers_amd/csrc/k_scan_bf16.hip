// k_scan_bf16.hip -- the selective scan's kernels for bf16 tensors (a file a type:
// they compile side by side).
#include "scan_grad_kernel.h"
#include "scan_kernel.h"

namespace rnnhip {

hipError_t launch_scan_local_bf16(const ScanArgs& a, hipStream_t s) { return scan_of<bf16_t, true>(a, s); }
hipError_t launch_scan_bf16(const ScanArgs& a, hipStream_t s) { return scan_of<bf16_t, false>(a, s); }
hipError_t launch_scan_backward_bf16(const ScanArgs& a, hipStream_t s) { return scan_backward_of<bf16_t>(a, s); }

}  // namespace rnnhip
