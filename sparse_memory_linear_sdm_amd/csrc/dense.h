// Launchers of the dense recurrence (linear*.hip) and the norms (norm.hip)
// behind the C ABI (host side).  Arguments are validated by the C-ABI layer
// (api_dense.hip) before any of these is called.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm {

// Steps per chunk of the dense recurrence: the products inside a chunk are
// taken on the matrix cores, the state is carried from chunk to chunk.  32 for
// fp32 (a chunk's tiles then take the LDS that 64 steps of bf16 take).
constexpr int linear_chunk(int dtype) { return dtype == 1 /* SDM_BF16 */ ? 64 : 32; }

// One call of the dense recurrence.  q, k [B, Hk, T, d_k]; v, out, dout
// [B, H, T, d_v]; g [B, H, T]; S, G [B, H, d_k, d_v].
struct LinearArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  void* out;
  float* S;      // forward: the state, in place; reverse: its gradient G
  float* tape;   // [B, H, chunks, d_k, d_v] states before each chunk, or null
  const void* dout;
  void* dq;
  void* dk;
  void* dv;
  float* dg;
  float* seg_state;  // [B, H, nseg, d_k, d_v] (nseg > 1)
  double* seg_log;   // [B, H, nseg] sums of log2 decays (nseg > 1)
  float* dq_part;    // [B, H, T, d_k] fp32 (shared keys)
  float* dk_part;
  int BH;      // memories
  int share;   // heads per key head, H / Hk
  int64_t T;
  int nchunk;
  int nseg;
  int seg_chunks;
};

// Up to this many segments, each adds up the states of those before it (behind
// it, in reverse) by itself; more are joined by a kernel of their own, since
// their states would be read too often (16 segments: 123 MB for 16 memories of
// 128 x 128).
constexpr int kOwnSegments = 8;

int linear_segments(int dtype, int64_t BH, int64_t T, int elems, bool backward);
size_t linear_scan_workspace_bytes(int dtype, int64_t BH, int d_k, int d_v, int64_t T);
size_t linear_backward_workspace_bytes(int dtype, int64_t BH, int share, int d_k, int d_v,
                                       int64_t T);
hipError_t launch_linear_scan(LinearArgs a, int dtype, int d_k, int d_v, void* ws,
                              hipStream_t stream);
hipError_t launch_linear_backward(LinearArgs a, int dtype, int d_k, int d_v, void* ws,
                                  hipStream_t stream);
hipError_t launch_linear_step(float* S, int dtype, int BH, int share, int d_k, int d_v,
                              const void* q, const void* k, const void* v, const float* g,
                              void* out, hipStream_t stream);

// The chunked kernels by type (linear_bf16.hip, linear_f32.hip; the reverse
// pass in linear_backward_*.hip).  mode: 0 the scan, 1 what each segment adds to
// the state, 2 the same for the state's gradient, segments and steps in reverse.
hipError_t launch_linear_bf16(const LinearArgs& a, int d_k, int d_v, int mode, hipStream_t stream);
hipError_t launch_linear_f32(const LinearArgs& a, int d_k, int d_v, int mode, hipStream_t stream);
hipError_t launch_linear_backward_bf16(const LinearArgs& a, int d_k, int d_v, hipStream_t stream);
hipError_t launch_linear_backward_f32(const LinearArgs& a, int d_k, int d_v, hipStream_t stream);

// Norm rows of d values (a multiple of 8, at most kNormMaxD).
constexpr int kNormMaxD = 16384;
struct NormDivisor {
  uint32_t mul;
  int shift;
  __device__ __forceinline__ uint32_t of(uint32_t n) const {
    return (uint32_t)((uint64_t)n * mul >> shift);
  }
};
struct NormArgs {
  const void* y;
  const float* w;
  const void* z;       // gate or null
  const void* x;       // residual or null
  float scale, eps;
  void* out;
  const float* next_w; // or null
  void* next;
  const void* dout;
  const void* skip;    // or null
  void* dy;
  void* dz;
  float* dw;
  float* part;         // [blocks, d] partial sums of dw
  int64_t rows;        // B * T * H
  int64_t T;
  int H, d;
  NormDivisor by_h, by_t;  // set by the launchers
};
hipError_t launch_norm(NormArgs a, int y_dtype, int out_dtype, hipStream_t stream);
int64_t norm_backward_blocks(int64_t rows, int d);
hipError_t launch_norm_backward(NormArgs a, int y_dtype, int out_dtype, hipStream_t stream);

}  // namespace sdm
