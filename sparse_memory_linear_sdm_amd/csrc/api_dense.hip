// C-ABI entry points of the dense recurrence and the norms: argument
// validation (before any launch) and dispatch to the kernels.
#include "../../include/sdm.h"
#include "api_common.h"
#include "dense.h"
#include "internal.h"

namespace {

using namespace sdm::api;

bool value_dtype(int dtype) { return dtype == SDM_F32 || dtype == SDM_BF16; }

bool head_supported(int d) { return d == 32 || d == 64 || d == 128; }

// One of a call's arrays: never NULL, `bytes` aligned.
int check_array(const void* p, size_t bytes, const char* name) {
  if (!p) return fail(SDM_ERR_INVALID, "%s is NULL", name);
  if (!aligned(p, bytes)) return fail(SDM_ERR_INVALID, "%s must be %zu-byte aligned", name, bytes);
  return SDM_OK;
}

int check_linear_sizes(int dtype, int B, int H, int Hk, int d_k, int d_v, int64_t T) {
  if (!value_dtype(dtype))
    return fail(SDM_ERR_INVALID, "dtype must be SDM_F32 or SDM_BF16 (got %d)", dtype);
  if (B < 1 || H < 1 || Hk < 1) return fail(SDM_ERR_INVALID, "B, H and Hk must be >= 1");
  if (H % Hk != 0) return fail(SDM_ERR_INVALID, "H must be a multiple of Hk (got %d, %d)", H, Hk);
  if ((int64_t)B * H > sdm::kMaxMemories)
    return fail(SDM_ERR_UNSUPPORTED, "B*H must be at most 2^20 memories per call");
  if (!head_supported(d_k)) return fail(SDM_ERR_UNSUPPORTED, "d_k=%d not compiled (32, 64, 128)", d_k);
  if (!head_supported(d_v)) return fail(SDM_ERR_UNSUPPORTED, "d_v=%d not compiled (32, 64, 128)", d_v);
  if (T < 0) return fail(SDM_ERR_INVALID, "T must be >= 0");
  if (T >= ((int64_t)1 << 31)) return fail(SDM_ERR_UNSUPPORTED, "T must be below 2^31");
  return SDM_OK;
}

// What the reverse pass takes, so that no tape is made that it would refuse.
int check_tape_steps(int B, int H, int64_t T) {
  if ((int64_t)B * H * T > sdm::kMaxWaveUnits)
    return fail(SDM_ERR_UNSUPPORTED, "B*H*T must be at most 2^26 - 4 per call with a tape");
  return SDM_OK;
}

int check_linear_inputs(const void* q, const void* k, const void* v, const float* g) {
  int rc;
  if ((rc = check_array(q, 16, "q")) || (rc = check_array(k, 16, "k")) ||
      (rc = check_array(v, 16, "v")) || (rc = check_array(g, 4, "g")))
    return rc;
  return SDM_OK;
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return SDM_OK;
  if (!ws) return fail(SDM_ERR_INVALID, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(SDM_ERR_INVALID, "workspace must be 256-byte aligned");
  if (bytes < need)
    return fail(SDM_ERR_INVALID, "workspace of %zu bytes is below the %zu required", bytes, need);
  return SDM_OK;
}

constexpr int64_t kNormRows = (int64_t)1 << 31;

bool norm_d_ok(int d) { return d >= 8 && d <= sdm::kNormMaxD && d % 8 == 0; }

bool norm_rows_ok(int B, int H, int64_t T) {
  return T < kNormRows && (int64_t)B * H < kNormRows && (int64_t)B * H * T < kNormRows;
}

int check_norm_sizes(int y_dtype, int out_dtype, float eps, int B, int H, int64_t T, int d) {
  if (!value_dtype(y_dtype) || !value_dtype(out_dtype))
    return fail(SDM_ERR_INVALID, "dtypes must be SDM_F32 or SDM_BF16 (got %d, %d)", y_dtype,
                out_dtype);
  if (B < 0 || H < 1 || T < 0) return fail(SDM_ERR_INVALID, "B and T must be >= 0 and H >= 1");
  if (!norm_d_ok(d))
    return fail(SDM_ERR_UNSUPPORTED, "d must be a multiple of 8 in [8, %d] (got %d)",
                sdm::kNormMaxD, d);
  if (!(eps >= 0.0f)) return fail(SDM_ERR_INVALID, "eps must be >= 0");
  if (!norm_rows_ok(B, H, T))
    return fail(SDM_ERR_UNSUPPORTED, "B*H*T must be below 2^31 rows per call");
  return SDM_OK;
}

}  // namespace

extern "C" {

size_t sdm_linear_scan_workspace_size(int dtype, int B, int H, int d_k, int d_v, int64_t T) {
  if (!value_dtype(dtype) || B < 1 || H < 1 || (int64_t)B * H > sdm::kMaxMemories ||
      !head_supported(d_k) || !head_supported(d_v) || T < 0 || T >= ((int64_t)1 << 31))
    return 0;
  return sdm::linear_scan_workspace_bytes(dtype, (int64_t)B * H, d_k, d_v, T);
}

int sdm_linear_scan(float* S, int dtype, int B, int H, int Hk, int d_k, int d_v, int64_t T,
                    const void* q, const void* k, const void* v, const float* g, void* out,
                    float* tape, void* workspace, size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = check_linear_sizes(dtype, B, H, Hk, d_k, d_v, T))) return rc;
  if (tape && (rc = check_tape_steps(B, H, T))) return rc;
  if ((rc = check_array(S, 16, "S"))) return rc;
  hipStream_t s = (hipStream_t)stream;
  if (T == 0) return finish("sdm_linear_scan", hipSuccess, s);  // the per-step arrays may be NULL
  if ((rc = check_linear_inputs(q, k, v, g))) return rc;
  if ((rc = check_array(out, 16, "out"))) return rc;
  if (!aligned(tape, 16)) return fail(SDM_ERR_INVALID, "tape must be 16-byte aligned");
  const size_t need = sdm::linear_scan_workspace_bytes(dtype, (int64_t)B * H, d_k, d_v, T);
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  sdm::LinearArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.out = out;
  a.S = S;
  a.tape = tape;
  a.BH = B * H;
  a.share = H / Hk;
  a.T = T;
  return finish("sdm_linear_scan", sdm::launch_linear_scan(a, dtype, d_k, d_v, workspace, s), s);
}

int sdm_linear_step(float* S, int dtype, int B, int H, int Hk, int d_k, int d_v, const void* q,
                    const void* k, const void* v, const float* g, void* out, void* stream) {
  int rc;
  if ((rc = check_linear_sizes(dtype, B, H, Hk, d_k, d_v, 1))) return rc;
  if ((rc = check_array(S, 16, "S")) || (rc = check_linear_inputs(q, k, v, g)) ||
      (rc = check_array(out, 16, "out")))
    return rc;
  hipStream_t s = (hipStream_t)stream;
  return finish("sdm_linear_step",
                sdm::launch_linear_step(S, dtype, B * H, H / Hk, d_k, d_v, q, k, v, g, out, s), s);
}

size_t sdm_linear_backward_workspace_size(int dtype, int B, int H, int Hk, int d_k, int d_v,
                                          int64_t T) {
  if (!value_dtype(dtype) || B < 1 || H < 1 || Hk < 1 || H % Hk != 0 ||
      (int64_t)B * H > sdm::kMaxMemories || !head_supported(d_k) || !head_supported(d_v) || T < 0 ||
      T > sdm::kMaxWaveUnits || (int64_t)B * H * T > sdm::kMaxWaveUnits)
    return 0;
  return sdm::linear_backward_workspace_bytes(dtype, (int64_t)B * H, H / Hk, d_k, d_v, T);
}

int sdm_linear_backward(int dtype, int B, int H, int Hk, int d_k, int d_v, int64_t T,
                        const void* q, const void* k, const void* v, const float* g,
                        const float* tape, const void* dout, float* G, void* dq, void* dk,
                        void* dv, float* dg, void* workspace, size_t workspace_bytes,
                        void* stream) {
  int rc;
  if ((rc = check_linear_sizes(dtype, B, H, Hk, d_k, d_v, T))) return rc;
  if ((rc = check_tape_steps(B, H, T))) return rc;
  if ((rc = check_array(G, 16, "G"))) return rc;
  hipStream_t s = (hipStream_t)stream;
  if (T == 0) return finish("sdm_linear_backward", hipSuccess, s);  // per-step arrays may be NULL
  if ((rc = check_linear_inputs(q, k, v, g))) return rc;
  if ((rc = check_array(tape, 16, "tape")) || (rc = check_array(dout, 16, "dout")) ||
      (rc = check_array(dq, 16, "dq")) || (rc = check_array(dk, 16, "dk")) ||
      (rc = check_array(dv, 16, "dv")) || (rc = check_array(dg, 4, "dg")))
    return rc;
  const size_t need =
      sdm::linear_backward_workspace_bytes(dtype, (int64_t)B * H, H / Hk, d_k, d_v, T);
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  sdm::LinearArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.S = G;
  a.tape = const_cast<float*>(tape);
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dg;
  a.BH = B * H;
  a.share = H / Hk;
  a.T = T;
  return finish("sdm_linear_backward", sdm::launch_linear_backward(a, dtype, d_k, d_v, workspace, s),
                s);
}

int sdm_norm(const void* y, int y_dtype, const float* w, const void* z, const void* x, float scale,
             float eps, int B, int H, int64_t T, int d, void* out, int out_dtype,
             const float* next_w, void* next, void* stream) {
  int rc;
  if ((rc = check_norm_sizes(y_dtype, out_dtype, eps, B, H, T, d))) return rc;
  if ((next_w == nullptr) != (next == nullptr))
    return fail(SDM_ERR_INVALID, "next_w and next come together");
  if (next && H != 1)
    return fail(SDM_ERR_INVALID, "next needs H = 1 (a row of out is one row of the next norm)");
  hipStream_t s = (hipStream_t)stream;
  const int64_t rows = (int64_t)B * H * T;
  if (rows == 0) return finish("sdm_norm", hipSuccess, s);  // the arrays may be NULL
  if ((rc = check_array(y, 16, "y")) || (rc = check_array(w, 16, "w")) ||
      (rc = check_array(out, 16, "out")))
    return rc;
  if (!aligned(z, 16) || !aligned(x, 16) || !aligned(next_w, 16) || !aligned(next, 16))
    return fail(SDM_ERR_INVALID, "z, x, next_w and next must be 16-byte aligned");
  sdm::NormArgs a = {};
  a.y = y;
  a.w = w;
  a.z = z;
  a.x = x;
  a.scale = scale;
  a.eps = eps;
  a.out = out;
  a.next_w = next_w;
  a.next = next;
  a.rows = rows;
  a.T = T;
  a.H = H;
  a.d = d;
  return finish("sdm_norm", sdm::launch_norm(a, y_dtype, out_dtype, s), s);
}

size_t sdm_norm_backward_workspace_size(int B, int H, int64_t T, int d) {
  if (B < 0 || H < 1 || T < 0 || !norm_d_ok(d) || !norm_rows_ok(B, H, T)) return 0;
  return (size_t)sdm::norm_backward_blocks((int64_t)B * H * T, d) * d * sizeof(float);
}

int sdm_norm_backward(const void* dout, int out_dtype, const void* y, int y_dtype, const float* w,
                      const void* z, const void* skip, float scale, float eps, int B, int H,
                      int64_t T, int d, void* dy, float* dw, void* dz, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = check_norm_sizes(y_dtype, out_dtype, eps, B, H, T, d))) return rc;
  if ((z == nullptr) != (dz == nullptr))
    return fail(SDM_ERR_INVALID, "z and dz come together");
  if ((rc = check_array(dw, 16, "dw"))) return rc;
  hipStream_t s = (hipStream_t)stream;
  const int64_t rows = (int64_t)B * H * T;
  if (rows > 0) {  // the other arrays may be NULL without rows
    if ((rc = check_array(dout, 16, "dout")) || (rc = check_array(y, 16, "y")) ||
        (rc = check_array(w, 16, "w")) || (rc = check_array(dy, 16, "dy")))
      return rc;
    if (!aligned(z, 16) || !aligned(dz, 16) || !aligned(skip, 16))
      return fail(SDM_ERR_INVALID, "z, dz and skip must be 16-byte aligned");
    const size_t need = (size_t)sdm::norm_backward_blocks(rows, d) * d * sizeof(float);
    if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  }
  sdm::NormArgs a = {};
  a.y = y;
  a.w = w;
  a.z = z;
  a.scale = scale;
  a.eps = eps;
  a.dout = dout;
  a.skip = skip;
  a.dy = dy;
  a.dz = dz;
  a.dw = dw;
  a.part = (float*)workspace;
  a.rows = rows;
  a.T = T;
  a.H = H;
  a.d = d;
  return finish("sdm_norm_backward", sdm::launch_norm_backward(a, y_dtype, out_dtype, s), s);
}

}  // extern "C"
