// Drives the microscaled entry points (csrc/api_mx.hip with csrc/api.hip,
// compiled host-only) under AddressSanitizer and UndefinedBehaviorSanitizer,
// with every kernel launcher replaced by a stub.  Checks: valid calls reach
// their launcher with the caller's sizes; invalid and extreme sizes are
// rejected before any launcher runs; launch errors map to SDM_ERR_HIP.
// Prints "ok" and exits 0 when every check passes.
#include <hip/hip_runtime_api.h>

#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/sdm.h"

namespace {
int g_launches = 0, g_fails = 0;
hipError_t g_launch_rc = hipSuccess;
long long g_last[7];

hipError_t record(long long a = 0, long long b = 0, long long c = 0, long long d = 0,
                  long long e = 0, long long f = 0, long long g = 0) {
  ++g_launches;
  const long long v[7] = {a, b, c, d, e, f, g};
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
uint8_t* const U = (uint8_t*)P;
float* const F = (float*)P;
int32_t* const I = (int32_t*)P;
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

hipError_t launch_mx4_quantize(const void*, int dtype, int64_t rows, int cols, uint8_t*, uint8_t*,
                               hipStream_t) {
  return record(dtype, rows, cols);
}
hipError_t launch_mx4_dequantize(const uint8_t*, const uint8_t*, int dtype, int64_t rows, int cols,
                                 void*, hipStream_t) {
  return record(dtype, rows, cols);
}
hipError_t launch_project_mx4(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*,
                              int B, int T, int d_model, int H, int n, int d_v, float*, float*,
                              float*, float*, float*, float*, float*, hipStream_t) {
  return record(B, T, d_model, H, n, d_v);
}
hipError_t launch_scan_train8(float*, int B, int H, int64_t N, int d_v, int64_t T, int W, int R,
                              const int32_t*, const float*, const int32_t*, const float*,
                              const float*, const float*, const float*, float*, int8_t*, uint8_t*,
                              hipStream_t) {
  return record(B, H, N, d_v, T, W, R);
}
hipError_t launch_tape8_read(const int8_t*, const uint8_t*, int dtype, int n_mem, int d_v,
                             int64_t S, void*, hipStream_t) {
  return record(dtype, n_mem, d_v, S);
}
hipError_t launch_scan_backward8(int B, int H, int64_t N, int d_v, int64_t T, int W, int R,
                                 const int32_t*, const float*, const int32_t*, const float*,
                                 const float*, const float*, const float*, const int8_t*,
                                 const uint8_t*, const float*, float*, float*, float*, float*,
                                 float*, float*, const uint64_t*, void*, hipStream_t) {
  return record(B, H, N, d_v, T, W, R);
}
size_t scan_backward8_workspace_bytes(int n_mem, int d_v, int64_t T, int W) {
  return (size_t)n_mem * (size_t)T * (size_t)(1296 + d_v / 16 * (W + 1) * 4);
}
}  // namespace sdm

namespace {
int train8(int B, int H, int64_t N, int d_v, int64_t T, int W, int R) {
  return sdm_scan_train8(P, B, H, N, d_v, T, W, R, I, F, I, F, F, F, F, F, (int8_t*)P, U, nullptr);
}
int backward8(int B, int H, int64_t N, int d_v, int64_t T, int W, int R, size_t bytes) {
  return sdm_scan_backward8(B, H, N, d_v, T, W, R, I, F, I, F, F, F, F, (int8_t*)P, U, F, F, F, F,
                            F, F, F, nullptr, P, bytes, nullptr);
}
int project(int B, int T, int d_model, int H, int n, int d_v) {
  return sdm_project_mx4(U, U, U, U, B, T, d_model, H, n, d_v, F, F, F, F, F, F, F, nullptr);
}
int read8(int B, int H, int d_v, int64_t T, int S) {
  return sdm_tape8_read((int8_t*)P, U, B, H, d_v, T, S, SDM_BF16, P, nullptr);
}
}  // namespace

int main() {
  int n = 0;
  CHECK(sdm_mx4_quantize(P, SDM_BF16, 12345, 640, U, U, nullptr) == SDM_OK && g_launches == ++n);
  CHECK(g_last[0] == SDM_BF16 && g_last[1] == 12345 && g_last[2] == 640);
  CHECK(sdm_mx4_dequantize(U, U, SDM_F32, 7, 65536, P, nullptr) == SDM_OK && g_launches == ++n);
  CHECK(project(3, 700, 256, 2, 37, 16) == SDM_OK && g_launches == ++n);
  CHECK(g_last[1] == 700 && g_last[4] == 37);
  CHECK(train8(2, 3, 4096, 128, 100, 64, 5) == SDM_OK && g_launches == ++n);
  CHECK(g_last[2] == 4096 && g_last[4] == 100 && g_last[6] == 5);
  CHECK(read8(2, 3, 256, 100, 128) == SDM_OK && g_launches == ++n);
  CHECK(g_last[1] == 6 && g_last[3] == 12800);
  const size_t ws = sdm_scan_backward8_workspace_size(2, 3, 128, 100, 64, 5);
  CHECK(backward8(2, 3, 4096, 128, 100, 64, 5, ws) == SDM_OK && g_launches == ++n);
  CHECK(backward8(2, 3, 4096, 128, 100, 64, 5, ws - 1) == SDM_ERR_INVALID);
  // the largest tape below 2 GiB, and the first one at it
  CHECK(train8(1, 1, 4096, 128, (1 << 17) - 1, 64, 64) == SDM_OK && g_launches == ++n);
  CHECK(train8(1, 1, 4096, 128, 1 << 17, 64, 64) == SDM_ERR_UNSUPPORTED);
  // extreme sizes
  const int64_t big[] = {INT64_MAX, INT64_MAX / 2, (int64_t)1 << 40, (int64_t)1 << 33};
  for (int64_t x : big) {
    CHECK(sdm_mx4_quantize(P, SDM_F32, x, 512, U, U, nullptr) == SDM_ERR_UNSUPPORTED);
    CHECK(sdm_mx4_quantize(P, SDM_F32, 4, x, U, U, nullptr) == SDM_ERR_UNSUPPORTED);
    CHECK(sdm_mx4_dequantize(U, U, SDM_F32, x, 512, P, nullptr) == SDM_ERR_UNSUPPORTED);
    CHECK(train8(1, 1, 4096, 128, x, 64, 64) == SDM_ERR_UNSUPPORTED);
    CHECK(backward8(1, 1, 4096, 128, x, 64, 64, SIZE_MAX) == SDM_ERR_UNSUPPORTED);
    CHECK(read8(1, 1, 256, x, 128) == SDM_ERR_UNSUPPORTED);
  }
  CHECK(project(INT_MAX, INT_MAX, 128, 1, 1, 1) == SDM_ERR_UNSUPPORTED);
  CHECK(project(1, 1, 128, INT_MAX, INT_MAX, INT_MAX) == SDM_ERR_UNSUPPORTED);
  CHECK(read8(INT_MAX, INT_MAX, 16, 1, 1) == SDM_ERR_UNSUPPORTED);
  CHECK(g_launches == n);
  // a launch error becomes SDM_ERR_HIP with the call's name
  g_launch_rc = hipErrorInvalidValue;
  CHECK(project(1, 1, 128, 1, 1, 1) == SDM_ERR_HIP && std::strstr(sdm_last_error(), "sdm_project_mx4"));
  CHECK(train8(1, 1, 64, 16, 1, 1, 1) == SDM_ERR_HIP && std::strstr(sdm_last_error(), "train8"));
  if (g_fails) return 1;
  std::puts("ok");
  return 0;
}
