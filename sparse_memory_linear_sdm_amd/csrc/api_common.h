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

inline bool dv_supported(int d) {
  return d == 16 || d == 32 || d == 64 || d == 128 || d == 256;
}

int check_project_sizes(int B, int T, int H, int n, int d_v);
int check_project_outputs(const float* s1, const float* s2, const float* q1, const float* q2,
                          const float* v, const float* alpha, const float* beta);


// The arguments of a scan over one state.
int check_scan_args(const void* M, int dtype, int B, int H, int64_t N, int d_v, int64_t T, int W,
                    int R, const int32_t* widx, const float* wk, const int32_t* ridx,
                    const float* rw, const float* v, const float* alpha, const float* beta,
                    const float* out);

// The arguments of a reverse pass from a tape of tape_elem bytes a value (4,
// or 1 for the 8-bit form); on success *need is its workspace in bytes.
int check_backward_args(int B, int H, int64_t N, int d_v, int64_t T, int W, int R,
                        const int32_t* widx, const float* wk, const int32_t* ridx,
                        const float* rw, const float* v, const float* alpha, const float* beta,
                        const void* tape, int tape_elem, const float* dout, float* G, float* dv,
                        float* dwk, float* drw, float* dalpha, float* dbeta,
                        const uint64_t* first, size_t* need);

}  // namespace api
}  // namespace sdm
