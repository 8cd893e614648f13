// C-ABI entry points of the microscaled operators: argument validation
// (before any launch) and dispatch to the kernels.
#include "../../include/sdm.h"
#include "api_common.h"
#include "internal.h"
#include "ranges.h"

namespace {

using namespace sdm::api;

// A 4-bit microscaled matrix and the type of its unquantised side.
int check_mx4(int64_t rows, int64_t cols, int dtype, int tile_cols, const uint8_t* codes,
              const uint8_t* scales) {
  if (dtype != SDM_F32 && dtype != SDM_BF16)
    return fail(SDM_ERR_INVALID, "dtype must be SDM_F32 or SDM_BF16 (got %d)", dtype);
  if (rows < 0) return fail(SDM_ERR_INVALID, "rows must be >= 0");
  if (cols < 128 || cols > 65536 || cols % 128 != 0)
    return fail(SDM_ERR_UNSUPPORTED, "cols must be a multiple of 128 in [128, 65536] (got %lld)",
                (long long)cols);
  if (rows >= ((int64_t)1 << 31) ||
      sdm::quantize_tiles(rows, (int)cols, tile_cols) > sdm::kMaxStrideBlocks)
    return fail(SDM_ERR_UNSUPPORTED, "rows must be below 2^31, and in at most 2^24 - 1 tiles of 8 "
                "rows x %d columns (rows=%lld, cols=%lld); split the rows over several calls",
                tile_cols, (long long)rows, (long long)cols);
  if (rows > 0 && (!codes || !scales))
    return fail(SDM_ERR_INVALID, "codes and scales must not be NULL");
  if (!aligned(codes, 16) || !aligned(scales, 4))
    return fail(SDM_ERR_INVALID, "codes must be 16-byte and scales 4-byte aligned");
  return SDM_OK;
}

}  // namespace

extern "C" {

int sdm_mx4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, uint8_t* codes,
                     uint8_t* scales, void* stream) {
  int rc;
  if ((rc = check_mx4(rows, cols, dtype, 512, codes, scales))) return rc;
  hipStream_t s = (hipStream_t)stream;
  if (rows == 0) return finish("sdm_mx4_quantize", hipSuccess, s);  // the arrays may be NULL
  if (!x) return fail(SDM_ERR_INVALID, "x is NULL");
  if (!aligned(x, 16)) return fail(SDM_ERR_INVALID, "x must be 16-byte aligned");
  return finish("sdm_mx4_quantize",
                sdm::launch_mx4_quantize(x, dtype, rows, (int)cols, codes, scales, s), s);
}

int sdm_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype, int64_t rows,
                       int64_t cols, void* x, void* stream) {
  int rc;
  const int tile_cols = sdm::dequantize_cols(dtype == SDM_BF16 ? 2 : 4);
  if ((rc = check_mx4(rows, cols, dtype, tile_cols, codes, scales))) return rc;
  hipStream_t s = (hipStream_t)stream;
  if (rows == 0) return finish("sdm_mx4_dequantize", hipSuccess, s);  // the arrays may be NULL
  if (!x) return fail(SDM_ERR_INVALID, "x is NULL");
  if (!aligned(x, 16)) return fail(SDM_ERR_INVALID, "x must be 16-byte aligned");
  return finish("sdm_mx4_dequantize",
                sdm::launch_mx4_dequantize(codes, scales, dtype, rows, (int)cols, x, s), s);
}

int sdm_project_mx4(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws,
                    int B, int T, int d_model, int H, int n, int d_v, float* s1, float* s2,
                    float* q1, float* q2, float* v, float* alpha, float* beta, void* stream) {
  if (d_model < 128 || d_model > 65536 || d_model % 128 != 0)
    return fail(SDM_ERR_UNSUPPORTED, "d_model must be a multiple of 128 in [128, 65536] (got %d)",
                d_model);
  int rc;
  if ((rc = check_project_sizes(B, T, H, n, d_v))) return rc;
  hipStream_t s = (hipStream_t)stream;
  if ((int64_t)B * T == 0) return finish("sdm_project_mx4", hipSuccess, s);  // arrays may be NULL
  if (!Xq || !Xs || !Wq || !Ws)
    return fail(SDM_ERR_INVALID, "Xq, Xs, Wq and Ws must not be NULL");
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Xs, 4) || !aligned(Ws, 4))
    return fail(SDM_ERR_INVALID, "codes must be 16-byte and scales 4-byte aligned");
  if ((rc = check_project_outputs(s1, s2, q1, q2, v, alpha, beta))) return rc;
  return finish("sdm_project_mx4",
                sdm::launch_project_mx4(Xq, Xs, Wq, Ws, B, T, d_model, H, n, d_v, s1, s2, q1, q2,
                                        v, alpha, beta, s), s);
}

int sdm_scan_train8(void* M, int B, int H, int64_t N, int d_v, int64_t T, int W, int R,
                    const int32_t* widx, const float* wk, const int32_t* ridx, const float* rw,
                    const float* v, const float* alpha, const float* beta, float* out,
                    int8_t* tape, uint8_t* tape_scale, void* stream) {
  int rc;
  if ((rc = check_scan_args(M, SDM_F32, B, H, N, d_v, T, W, R, widx, wk, ridx, rw, v, alpha,
                            beta, out)))
    return rc;
  if (T > 0 && (!tape || !tape_scale))
    return fail(SDM_ERR_INVALID, "tape and tape_scale must not be NULL");
  if (!aligned(tape, 16)) return fail(SDM_ERR_INVALID, "tape must be 16-byte aligned");
  if (T * (W + R) * d_v >= ((int64_t)1 << 31))
    return fail(SDM_ERR_UNSUPPORTED, "one memory's tape (T*(W+R)*d_v bytes) must be below 2 GiB; "
                "split the sequence into consecutive calls");
  if (!sdm::ranges::tape8_ok(d_v, T, W, R))
    return fail(SDM_ERR_UNSUPPORTED, "a tape buffer range does not fit 31 bits");
  hipStream_t s = (hipStream_t)stream;
  return finish("sdm_scan_train8",
                sdm::launch_scan_train8(reinterpret_cast<float*>(M), B, H, N, d_v, T, W, R, widx,
                                        wk, ridx, rw, v, alpha, beta, out, tape, tape_scale, s),
                s);
}

int sdm_tape8_read(const int8_t* tape, const uint8_t* tape_scale, int B, int H, int d_v,
                   int64_t T, int S, int dtype, void* rows, void* stream) {
  if (B < 1 || H < 1) return fail(SDM_ERR_INVALID, "B and H must be >= 1");
  if ((int64_t)B * H > sdm::kMaxMemories)
    return fail(SDM_ERR_UNSUPPORTED, "B*H must be at most 2^20 memories per call");
  if (!dv_supported(d_v))
    return fail(SDM_ERR_UNSUPPORTED, "d_v=%d not compiled (16, 32, 64, 128, 256)", d_v);
  if (dtype != SDM_F32 && dtype != SDM_BF16)
    return fail(SDM_ERR_INVALID, "dtype must be SDM_F32 or SDM_BF16 (got %d)", dtype);
  if (T < 0) return fail(SDM_ERR_INVALID, "T must be >= 0");
  if (S < 1 || S > 128) return fail(SDM_ERR_INVALID, "S (rows per step, W + R) must be in [1, 128]");
  if (T >= ((int64_t)1 << 31) || T * S * d_v >= ((int64_t)1 << 31))
    return fail(SDM_ERR_UNSUPPORTED, "one memory's tape (T*S*d_v bytes) must be below 2 GiB");
  hipStream_t s = (hipStream_t)stream;
  if (T == 0) return finish("sdm_tape8_read", hipSuccess, s);  // the arrays may be NULL
  if (!tape || !tape_scale || !rows)
    return fail(SDM_ERR_INVALID, "tape, tape_scale and rows must not be NULL");
  if (!aligned(tape, 16) || !aligned(rows, 16))
    return fail(SDM_ERR_INVALID, "tape and rows must be 16-byte aligned");
  return finish("sdm_tape8_read",
                sdm::launch_tape8_read(tape, tape_scale, dtype, B * H, d_v, T * S, rows, s), s);
}

size_t sdm_scan_backward8_workspace_size(int B, int H, int d_v, int64_t T, int W, int R) {
  if (B < 1 || H < 1 || T < 0 || W < 1 || W > 64 || R < 1 || R > 64 || !dv_supported(d_v)) return 0;
  if ((int64_t)B * H > sdm::kMaxMemories || T > sdm::kMaxWaveUnits) return 0;
  // the call's own limits on the steps and on one memory's tape
  if ((int64_t)B * H * (T + sdm::kBackward8Pad) > sdm::kMaxWaveUnits ||
      T * (W + R) * d_v >= ((int64_t)1 << 31) || !sdm::ranges::tape8_ok(d_v, T, W, R))
    return 0;
  return sdm::scan_backward8_workspace_bytes(B * H, d_v, T, W);
}

int sdm_scan_backward8(int B, int H, int64_t N, int d_v, int64_t T, int W, int R,
                       const int32_t* widx, const float* wk, const int32_t* ridx,
                       const float* rw, const float* v, const float* alpha, const float* beta,
                       const int8_t* tape, const uint8_t* tape_scale, const float* dout, float* G,
                       float* dv, float* dwk, float* drw, float* dalpha, float* dbeta,
                       const uint64_t* first, void* workspace, size_t workspace_bytes,
                       void* stream) {
  int rc;
  size_t need = 0;  // of the other reverse pass
  if ((rc = check_backward_args(B, H, N, d_v, T, W, R, widx, wk, ridx, rw, v, alpha, beta, tape, 1,
                                dout, G, dv, dwk, drw, dalpha, dbeta, first, &need)))
    return rc;
  if ((int64_t)B * H * (T + sdm::kBackward8Pad) > sdm::kMaxWaveUnits)
    return fail(SDM_ERR_UNSUPPORTED,
                "B*H*(T + 8) must be at most 2^26 - 4 (one wavefront per memory and step)");
  need = T > 0 ? sdm::scan_backward8_workspace_bytes(B * H, d_v, T, W) : 0;
  if (T > 0 && !tape_scale) return fail(SDM_ERR_INVALID, "tape_scale is NULL");
  if (T > 0 && !workspace) return fail(SDM_ERR_INVALID, "workspace is NULL");
  if (!aligned(workspace, 16)) return fail(SDM_ERR_INVALID, "workspace must be 16-byte aligned");
  if (workspace_bytes < need)
    return fail(SDM_ERR_INVALID, "workspace of %zu bytes is below the %zu required",
                workspace_bytes, need);
  hipStream_t s = (hipStream_t)stream;
  return finish("sdm_scan_backward8",
                sdm::launch_scan_backward8(B, H, N, d_v, T, W, R, widx, wk, ridx, rw, v, alpha,
                                           beta, tape, tape_scale, dout, G, dv, dwk, drw, dalpha,
                                           dbeta, first, workspace, s),
                s);
}

}  // extern "C"
