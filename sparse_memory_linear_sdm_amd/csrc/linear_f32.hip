// Chunked kernels of the dense recurrence (linear_scan.h) for fp32.
#include "linear_scan.h"

namespace sdm {
hipError_t launch_linear_f32(const LinearArgs& a, int d_k, int d_v, int mode, hipStream_t stream) {
  return lin::launch_scan_type<float>(a, d_k, d_v, mode, stream);
}
}  // namespace sdm
