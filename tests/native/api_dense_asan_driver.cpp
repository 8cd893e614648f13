// Drives the entry points of the dense recurrence and the norms
// (csrc/api_dense.hip with csrc/api.hip, compiled host-only) under
// AddressSanitizer and UndefinedBehaviorSanitizer, with every kernel launcher
// replaced by a stub.  Checks: valid calls reach their launcher with the
// caller's sizes; invalid and extreme sizes are rejected before any launcher
// runs; launch errors map to SDM_ERR_HIP.  Prints "ok" and exits 0 when every
// check passes.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/sdm.h"
#include "../../sparse_memory_linear_sdm_amd/csrc/dense.h"

namespace {
int g_launches = 0, g_fails = 0;
hipError_t g_launch_rc = hipSuccess;
long long g_last[6];

hipError_t record(long long a = 0, long long b = 0, long long c = 0, long long d = 0,
                  long long e = 0, long long f = 0) {
  ++g_launches;
  const long long v[6] = {a, b, c, d, e, f};
  std::memcpy(g_last, v, sizeof v);
  return g_launch_rc;
}

void check(bool ok, const char* what, int line) {
  if (!ok) {
    std::fprintf(stderr, "FAIL line %d: %s (last error: %s)\n", line, what, sdm_last_error());
    ++g_fails;
  }
}
#define CHECK(x) check((x), #x, __LINE__)

void* const P = (void*)(uintptr_t)(1 << 20);  // aligned, never dereferenced
float* const F = (float*)P;
}  // namespace

extern "C" {
const char* hipGetErrorString(hipError_t) { return "stub error"; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
}

// The launchers of api.hip are linked but not reached here.
namespace sdm {
#define NOT_REACHED return record(-1)
hipError_t launch_project(const uint16_t*, const uint16_t*, int, int, int, int, int, int, float*,
                          float*, float*, float*, float*, float*, float*, hipStream_t) {
  NOT_REACHED;
}
hipError_t launch_select(const float*, const float*, int64_t, int, int, int32_t*, float*, float*,
                         hipStream_t) {
  NOT_REACHED;
}
hipError_t launch_state_init(void*, int, const float*, int, int, int64_t, int, hipStream_t) {
  NOT_REACHED;
}
hipError_t launch_scan(void*, int, int, int, int64_t, int, int64_t, int, int, const int32_t*,
                       const float*, const int32_t*, const float*, const float*, const float*,
                       const float*, float*, void*, hipStream_t) {
  NOT_REACHED;
}
hipError_t launch_step_decode(void*, int, int, int, int, int, int, int, const float*, const float*,
                              const float*, const float*, const float*, const float*, const float*,
                              float*, int32_t*, int32_t*, hipStream_t) {
  NOT_REACHED;
}
size_t scan_backward_workspace_bytes(int n_mem, int d_v, int64_t T, int W, int R) {
  return (size_t)n_mem * (size_t)T * (size_t)(d_v / 16) * (size_t)(W + R + 1) * 4;
}
hipError_t launch_scan_backward(int, int, int64_t, int, int64_t, int, int, const int32_t*,
                                const float*, const int32_t*, const float*, const float*,
                                const float*, const float*, const float*, const float*, float*,
                                float*, float*, float*, float*, float*, const uint64_t*, float*,
                                hipStream_t) {
  NOT_REACHED;
}
hipError_t static_scratch(void** ptr) {
  *ptr = nullptr;
  NOT_REACHED;
}
hipError_t launch_select_backward(const int32_t*, const float*, const float*, int64_t, int, int,
                                  float*, float*, hipStream_t) {
  NOT_REACHED;
}
hipError_t launch_state_init_backward(const float*, int, int, int64_t, int, const uint32_t*,
                                      float*, hipStream_t) {
  NOT_REACHED;
}
hipError_t launch_touch_prepare(int, int, int64_t, int64_t, int, int, const int32_t*,
                                const int32_t*, uint32_t*, uint64_t*, hipStream_t) {
  NOT_REACHED;
}
int planned_shards(int, int) { return 1; }
hipError_t launch_scan_plan(int, int, int64_t, int, int64_t, int, int, const int32_t*,
                            const float*, const int32_t*, const float*, void*, hipStream_t) {
  NOT_REACHED;
}
hipError_t launch_scan_planned(float*, int, int, int64_t, int, int64_t, const float*, const float*,
                               const float*, float*, void*, hipStream_t) {
  NOT_REACHED;
}

size_t linear_scan_workspace_bytes(int, int64_t BH, int d_k, int d_v, int64_t T) {
  return T > 512 ? (size_t)BH * d_k * d_v * 4 : 0;
}
size_t linear_backward_workspace_bytes(int, int64_t BH, int share, int d_k, int, int64_t T) {
  return share > 1 ? (size_t)BH * T * d_k * 8 : 0;
}
int64_t norm_backward_blocks(int64_t rows, int) { return rows < 512 ? rows : 512; }
hipError_t launch_linear_scan(LinearArgs a, int dtype, int d_k, int d_v, void*, hipStream_t) {
  return record(dtype, a.BH, a.share, d_k, d_v, a.T);
}
hipError_t launch_linear_backward(LinearArgs a, int dtype, int d_k, int d_v, void*, hipStream_t) {
  return record(dtype, a.BH, a.share, d_k, d_v, a.T);
}
hipError_t launch_linear_step(float*, int dtype, int BH, int share, int d_k, int d_v, const void*,
                              const void*, const void*, const float*, void*, hipStream_t) {
  return record(dtype, BH, share, d_k, d_v);
}
hipError_t launch_norm(NormArgs a, int y, int out, hipStream_t) {
  return record(y, out, a.rows, a.T, a.H, a.d);
}
hipError_t launch_norm_backward(NormArgs a, int y, int out, hipStream_t) {
  return record(y, out, a.rows, a.T, a.H, a.d);
}
}  // namespace sdm

namespace {
int scan(int B, int H, int Hk, int dk, int dv, int64_t T, size_t bytes = SIZE_MAX) {
  return sdm_linear_scan(F, SDM_BF16, B, H, Hk, dk, dv, T, P, P, P, F, P, F, P, bytes, nullptr);
}
int step(int B, int H, int Hk, int dk, int dv) {
  return sdm_linear_step(F, SDM_F32, B, H, Hk, dk, dv, P, P, P, F, P, nullptr);
}
int backward(int B, int H, int Hk, int dk, int dv, int64_t T, size_t bytes = SIZE_MAX) {
  return sdm_linear_backward(SDM_F32, B, H, Hk, dk, dv, T, P, P, P, F, F, P, F, P, P, P, F, P,
                             bytes, nullptr);
}
int norm(int B, int H, int64_t T, int d) {
  return sdm_norm(P, SDM_F32, F, P, P, 0.5f, 1e-6f, B, H, T, d, P, SDM_BF16, nullptr, nullptr,
                  nullptr);
}
int norm_backward(int B, int H, int64_t T, int d, size_t bytes = SIZE_MAX) {
  return sdm_norm_backward(P, SDM_BF16, P, SDM_F32, F, P, P, 0.5f, 1e-6f, B, H, T, d, P, F, P, P,
                           bytes, nullptr);
}
}  // namespace

int main() {
  int n = 0;
  CHECK(scan(2, 6, 3, 64, 128, 1000) == SDM_OK && g_launches == ++n);
  CHECK(g_last[1] == 12 && g_last[2] == 2 && g_last[3] == 64 && g_last[4] == 128 && g_last[5] == 1000);
  const size_t ws = sdm_linear_scan_workspace_size(SDM_BF16, 2, 6, 64, 128, 1000);
  CHECK(ws == 12u * 64 * 128 * 4);
  CHECK(scan(2, 6, 3, 64, 128, 1000, ws) == SDM_OK && g_launches == ++n);
  CHECK(scan(2, 6, 3, 64, 128, 1000, ws - 1) == SDM_ERR_INVALID);
  CHECK(scan(2, 6, 3, 64, 128, 0, 0) == SDM_OK);
  CHECK(step(1 << 10, 1 << 10, 1, 32, 32) == SDM_OK && g_launches == ++n && g_last[1] == 1 << 20);
  CHECK(backward(2, 4, 2, 32, 64, 77) == SDM_OK && g_launches == ++n && g_last[2] == 2);
  CHECK(backward(2, 4, 2, 32, 64, 77, 8u * 77 * 32 * 8 - 1) == SDM_ERR_INVALID);
  CHECK(backward(1, 1, 1, 32, 32, (1 << 26) - 4) == SDM_OK && g_launches == ++n);
  CHECK(backward(1, 1, 1, 32, 32, (1 << 26) - 3) == SDM_ERR_UNSUPPORTED);
  CHECK(norm(3, 5, 7, 16384) == SDM_OK && g_launches == ++n && g_last[2] == 105);
  CHECK(norm(0, 5, 7, 16384) == SDM_OK);
  CHECK(norm(1, 1, (1ll << 31) - 1, 8) == SDM_OK && g_launches == ++n);
  CHECK(norm_backward(3, 5, 7, 24) == SDM_OK && g_launches == ++n);
  CHECK(norm_backward(3, 5, 7, 24, sdm_norm_backward_workspace_size(3, 5, 7, 24) - 1) == SDM_ERR_INVALID);
  CHECK(norm_backward(3, 5, 0, 24, 0) == SDM_OK && g_launches == ++n);  // dw = 0
  // extreme sizes
  const int64_t big[] = {INT64_MAX, INT64_MAX / 2, (int64_t)1 << 40, (int64_t)1 << 31};
  for (int64_t x : big) {
    CHECK(scan(1, 1, 1, 32, 32, x) == SDM_ERR_UNSUPPORTED);
    CHECK(backward(1, 1, 1, 32, 32, x) == SDM_ERR_UNSUPPORTED);
    CHECK(norm(1, 1, x, 8) == SDM_ERR_UNSUPPORTED);
    CHECK(norm_backward(1, 1, x, 8) == SDM_ERR_UNSUPPORTED);
    CHECK(sdm_linear_scan_workspace_size(SDM_F32, 1, 1, 32, 32, x) == 0);
    CHECK(sdm_linear_backward_workspace_size(SDM_F32, 1, 1, 1, 32, 32, x) == 0);
    CHECK(sdm_norm_backward_workspace_size(1, 1, x, 8) == 0);
  }
  CHECK(scan(INT_MAX, INT_MAX, 1, 32, 32, 1) == SDM_ERR_UNSUPPORTED);
  CHECK(step(INT_MAX, INT_MAX, INT_MAX, 32, 32) == SDM_ERR_UNSUPPORTED);
  CHECK(norm(INT_MAX, INT_MAX, INT_MAX, 8) == SDM_ERR_UNSUPPORTED);
  CHECK(norm_backward(INT_MAX, INT_MAX, 1, 8) == SDM_ERR_UNSUPPORTED);
  CHECK(norm(INT_MIN, 1, 1, 8) == SDM_ERR_INVALID && scan(INT_MIN, 1, 1, 32, 32, 1) == SDM_ERR_INVALID);
  CHECK(g_launches == n);
  // a launch error becomes SDM_ERR_HIP with the call's name
  g_launch_rc = hipErrorInvalidValue;
  CHECK(step(1, 1, 1, 32, 32) == SDM_ERR_HIP && std::strstr(sdm_last_error(), "sdm_linear_step"));
  CHECK(norm(1, 1, 1, 8) == SDM_ERR_HIP && std::strstr(sdm_last_error(), "sdm_norm"));
  if (g_fails) return 1;
  std::puts("ok");
  return 0;
}
