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
  float* dst;  // NULL past the last column
  int64_t stride;  // elements per token of the destination
  int off, h;
  bool gate;
};

// (columns are below 2^31: 32-bit divisions)
__device__ __forceinline__ ProjColumn project_column(const ProjOut& A, uint32_t col) {
  ProjColumn c = {};
  if (col >= (uint32_t)A.Ncols) return c;
  c.h = (int)(col / (uint32_t)A.P);
  const int p = (int)(col - (uint32_t)c.h * (uint32_t)A.P);
  if (p < 4 * A.n) {
    const int part = (int)((uint32_t)p / (uint32_t)A.n);
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

// One value of a token (b, t); tok = b*H*T + t.
__device__ __forceinline__ void project_store_one(const ProjOut& A, const ProjColumn& c,
                                                  int64_t tok, float y) {
  c.dst[(tok + (int64_t)c.h * A.T) * c.stride + c.off] = c.gate ? sigmoidf_(y) : y;
}

__device__ __forceinline__ int64_t project_token(const ProjOut& A, uint32_t row) {
  const uint32_t b = row / (uint32_t)A.T;
  return (int64_t)b * A.H * A.T + (row - b * (uint32_t)A.T);
}

// A wavefront's NJ neighbouring 32 x 32 accumulator blocks: value r of block j
// is column c[j]'s token row0 + 8*(r/4) + 4*(lane/32) + r%4.  A token's
// columns go out together, so that the pieces of a cache line, which the
// columns' offsets seldom start at, meet in L2.  Where the 32 tokens are of
// one sequence and no column is a gate or past the end, an address is the
// last one plus a multiple of its column's stride; else each token is found
// by a division (tokens < 2^32).  (Stepping token by token with its checks,
// for all, took 20 us per 256 x 256 tile, a seventh of the product's time at
// d_model 16384.)
template <int NJ>
__device__ __forceinline__ void project_store_blocks(const ProjOut& A, const ProjColumn (&c)[NJ],
                                                     int64_t row0, const f32x16 (&acc)[NJ]) {
  if (row0 >= A.M) return;
  const int lh = lane_id() >> 5;
  const uint32_t t0 = (uint32_t)row0 % (uint32_t)A.T;
  bool plain = true;
#pragma unroll
  for (int j = 0; j < NJ; ++j) plain = plain && c[j].dst && !c[j].gate;
  if (row0 + 32 <= A.M && t0 + 32 <= (uint32_t)A.T && __all(plain)) {
    const int64_t tok = project_token(A, (uint32_t)row0) + 4 * lh;
    float* p[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) p[j] = c[j].dst + (tok + (int64_t)c[j].h * A.T) * c[j].stride + c[j].off;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        *p[j] = acc[j][r];
        p[j] += (r & 3) == 3 ? 5 * c[j].stride : c[j].stride;  // rows 0,1,2,3, 8,9,10,11, 16,...
      }
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t row = row0 + 8 * (r >> 2) + 4 * lh + (r & 3);
    if (row >= A.M) continue;
    const int64_t tok = project_token(A, (uint32_t)row);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (c[j].dst) project_store_one(A, c[j], tok, acc[j][r]);
  }
}

// 64 tokens' values of a wavefront's 64 columns, one column a lane: token
// row0 + r's at y[r * kWave ..] (the wavefront's own LDS; changed).
__device__ __forceinline__ void project_store_rows(const ProjOut& A, const ProjColumn& c,
                                                   int64_t row0, float* y) {
  constexpr int kEach = 8;  // rows read together
  const int rows = A.M - row0 < kWave ? (int)(A.M - row0) : kWave;
  if (rows <= 0) return;
  const int lane = lane_id();
  // gate columns, one after the other with a token a lane: their few values a
  // row would cost every row the logistic function's instructions
  for (uint64_t m = __ballot(c.gate); m; m &= m - 1) {
    float& g = y[lane * kWave + __builtin_ctzll(m)];
    g = sigmoidf_(g);
  }
  wave_sync();
  if (!c.dst) return;
  // Which token comes next is the same for every lane, so an address is the
  // last one plus the column's stride, and a step over the other heads at the
  // end of a sequence.
  const uint32_t T = (uint32_t)A.T;
  uint32_t t = (uint32_t)row0 % T;
  const bool whole = rows == kWave && t + kWave <= T;  // all of one sequence
  const int64_t over = (int64_t)(A.H - 1) * A.T * c.stride;
  float* p = c.dst + (project_token(A, (uint32_t)row0) + (int64_t)c.h * A.T) * c.stride + c.off;
#pragma unroll 1
  for (int r = 0; r < rows; r += kEach) {
    float v[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) v[u] = y[(r + u) * kWave + lane];
    if (whole) {
#pragma unroll
      for (int u = 0; u < kEach; ++u, p += c.stride) *p = v[u];
      continue;
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      if (r + u >= rows) break;
      *p = v[u];
      p += c.stride;
      if (++t == T) {
        t = 0;
        p += over;
      }
    }
  }
}

}  // namespace sdm
