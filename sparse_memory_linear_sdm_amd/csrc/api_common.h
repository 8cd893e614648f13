// What the files of C-ABI entry points share (defined in api.hip): the error
// text of the calling thread, the end of a call, and argument checks that
// several calls need.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm {
namespace api {

// Record the calling thread's error text and return the status.
int fail(int status, const char* fmt, ...);

// The status of a call whose launches returned launch_err (waits for the
// stream when SDM_DEBUG_SYNC=1).
int finish(const char* what, hipError_t launch_err, hipStream_t stream);

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_project_sizes(int B, int T, int H, int n, int d_v);
int check_project_outputs(const float* s1, const float* s2, const float* q1, const float* q2,
                          const float* v, const float* alpha, const float* beta);

}  // namespace api
}  // namespace sdm
