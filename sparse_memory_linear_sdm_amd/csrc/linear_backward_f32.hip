// Reverse pass of the dense recurrence (linear_backward.h) for fp32.
#include "linear_backward.h"

namespace sdm {
hipError_t launch_linear_backward_f32(const LinearArgs& a, int d_k, int d_v, hipStream_t stream) {
  return lin::launch_backward_type<float>(a, d_k, d_v, stream);
}
}  // namespace sdm
