// C-ABI entry points of the microscaled operators: argument validation
// (before any launch) and dispatch to the kernels.
#include "../../include/sdm.h"
#include "api_common.h"
#include "internal.h"

namespace {

using namespace sdm::api;

// A 4-bit microscaled matrix and the type of its unquantised side.
int check_mx4(int64_t rows, int64_t cols, int dtype, const uint8_t* codes, const uint8_t* scales) {
  if (dtype != SDM_F32 && dtype != SDM_BF16)
    return fail(SDM_ERR_INVALID, "dtype must be SDM_F32 or SDM_BF16 (got %d)", dtype);
  if (rows < 0) return fail(SDM_ERR_INVALID, "rows must be >= 0");
  if (cols < 128 || cols > 65536 || cols % 128 != 0)
    return fail(SDM_ERR_UNSUPPORTED, "cols must be a multiple of 128 in [128, 65536] (got %lld)",
                (long long)cols);
  if (rows >= ((int64_t)1 << 31) ||
      sdm::quantize_blocks(rows, (int)cols) > sdm::kMaxStrideBlocks)
    return fail(SDM_ERR_UNSUPPORTED, "more than 2^24 - 1 tiles of 32 rows x 512 columns "
                "(rows=%lld, cols=%lld); split the rows over several calls", (long long)rows,
                (long long)cols);
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
  if ((rc = check_mx4(rows, cols, dtype, codes, scales))) return rc;
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
  if ((rc = check_mx4(rows, cols, dtype, codes, scales))) return rc;
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

}  // extern "C"
