// Where the projections' values go: s1, s2, q1, q2 [B, H, T, n], v
// [B, H, T, d_v] and the gates [B, H, T] (token m = b*T + t, column
// h*P + p with P = 4n + d_v + 2), the layouts the selection and the scan read.
#pragma once
#include "device_common.h"

namespace sdm {

typedef float f32x16 __attribute__((ext_vector_type(16)));

struct ProjOut {
  int64_t M;  // tokens, B * T
  int H, P, n, d_v, T;
  int64_t Ncols;  // H * P
  float *s1, *s2, *q1, *q2, *v, *alpha, *beta;
};

inline ProjOut project_out(int B, int T, int H, int n, int d_v, float* s1, float* s2, float* q1,
                           float* q2, float* v, float* alpha, float* beta) {
  const int P = 4 * n + d_v + 2;
  return ProjOut{(int64_t)B * T, H, P, n, d_v, T, (int64_t)H * P, s1, s2, q1, q2, v, alpha, beta};
}

__device__ __forceinline__ float sigmoidf_(float y) { return 1.0f / (1.0f + expf(-y)); }

// The array, token stride and offset of one column.
struct ProjColumn {
  float* dst;
  int64_t stride;  // elements per token of the destination
  int off, h;
  bool gate;
};

__device__ __forceinline__ ProjColumn project_column(const ProjOut& A, int64_t col) {
  ProjColumn c;
  c.h = (int)(col / A.P);
  const int p = (int)(col % A.P);
  c.gate = false;
  if (p < 4 * A.n) {
    const int part = p / A.n;
    c.dst = part == 0 ? A.s1 : part == 1 ? A.s2 : part == 2 ? A.q1 : A.q2;
    c.stride = A.n;
    c.off = p - part * A.n;
  } else if (p < 4 * A.n + A.d_v) {
    c.dst = A.v;
    c.stride = A.d_v;
    c.off = p - 4 * A.n;
  } else {
    c.dst = p == 4 * A.n + A.d_v ? A.alpha : A.beta;
    c.stride = 1;
    c.off = 0;
    c.gate = true;
  }
  return c;
}

// One lane's part of a 32 x 32 accumulator block: value r is the column's
// token rb + 8*(r/4) + r%4 (rb: the block's first token + 4 * (lane / 32)).
// The token (b, t) of rb by one division (tokens < 2^32), then stepped.
__device__ __forceinline__ void project_store_block(const ProjOut& A, const ProjColumn& c,
                                                    int64_t rb, const f32x16& acc) {
  if (rb >= A.M) return;
  const int64_t HT = (int64_t)A.H * A.T;
  uint32_t b = (uint32_t)rb / (uint32_t)A.T, t = (uint32_t)rb - b * (uint32_t)A.T;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (r > 0) {
      t += (r & 3) ? 1 : 5;  // the row offsets run 0,1,2,3, 8,9,10,11, 16,...
      while (t >= (uint32_t)A.T) {
        t -= (uint32_t)A.T;
        ++b;
      }
    }
    const int64_t row = rb + 8 * (r >> 2) + (r & 3);
    if (row >= A.M) break;
    const int64_t tok = (int64_t)b * HT + (int64_t)c.h * A.T + t;  // ((b*H + h)*T + t)
    const float y = acc[r];
    c.dst[tok * c.stride + c.off] = c.gate ? sigmoidf_(y) : y;
  }
}

// One value.
__device__ __forceinline__ void project_store_one(const ProjOut& A, const ProjColumn& c,
                                                  int64_t row, float y) {
  const uint32_t b = (uint32_t)row / (uint32_t)A.T, t = (uint32_t)row - b * (uint32_t)A.T;
  const int64_t tok = ((int64_t)b * A.H + c.h) * A.T + t;
  c.dst[tok * c.stride + c.off] = c.gate ? sigmoidf_(y) : y;
}

}  // namespace sdm
