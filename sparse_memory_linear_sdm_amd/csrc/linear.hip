// The dense recurrence with a decay for each head: the host side of the chunked
// kernels, the sums over segments and over heads that share keys, and the step
// of a single token.
#include "dense.h"
#include "linear_tile.h"

namespace sdm {
namespace {

constexpr int kThreads = 256;

// What each segment starts from: the call's state carried through the
// segments before it (behind it, in reverse).  seg_state[m][i] holds what
// segment i adds; afterwards what it starts from.  A thread takes four values
// of kPer consecutive segments; kGroups threads share a memory's segments, and
// carry the state over each other's by sums and decays in LDS.  Bound by memory:
// 32 segments of 16 memories of 128 x 128 (67 MB) 11 us.  (One thread through 128
// segments of 4 memories took 45 us.)
template <int kGroups, int kPer>
__global__ __launch_bounds__(kThreads) void linear_segments_kernel(float* seg_state,
                                                                   const double* seg_log,
                                                                   const float* S, int64_t total,
                                                                   int elems, int nseg,
                                                                   bool reverse) {
  constexpr int kLanes = kThreads / kGroups;
  __shared__ f32x4 sums[kGroups][kLanes];
  __shared__ float decays[kGroups][kLanes];
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int64_t at = ((int64_t)blockIdx.x * kLanes + lane) * 4;  // whole workgroups: total is
  const int64_t m = at / elems, e = at % elems;                  // a multiple of 4 kLanes
  f32x4 run = *reinterpret_cast<const f32x4*>(S + at);
  float* p = seg_state + m * nseg * elems + e;
  const double* lg = seg_log + m * nseg;
  const int i0 = group * kPer;
  f32x4 own[kPer];
  float decay[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = reverse ? nseg - 1 - (i0 + j) : i0 + j;
    own[j] = f32x4{0, 0, 0, 0};
    decay[j] = 1.0f;
    if (i0 + j < nseg - 1) {  // the last of the order passes nothing on
      own[j] = *reinterpret_cast<const f32x4*>(p + (int64_t)i * elems);
      decay[j] = lin::pow2((float)lg[i]);
    }
  }
  f32x4 sum = own[0];
  float d = decay[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) {
    sum = sum * decay[j] + own[j];
    d *= decay[j];
  }
  sums[group][lane] = sum;
  decays[group][lane] = d;
  __syncthreads();
  for (int i = 0; i < group; ++i) run = run * decays[i][lane] + sums[i][lane];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = reverse ? nseg - 1 - (i0 + j) : i0 + j;
    if (i0 + j < nseg) *reinterpret_cast<f32x4*>(p + (int64_t)i * elems) = run;
    run = run * decay[j] + own[j];
  }
}

// Gradients of shared keys: the sum over the heads that share them, in their
// order, rounded once (one pass over the parts, bound by memory).  blockIdx.y:
// dq, dk.
template <class T>
__global__ __launch_bounds__(kThreads) void linear_share_kernel(LinearArgs A, int64_t total,
                                                                int64_t per_head) {
  const int64_t at = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  if (at >= total) return;
  const float* p = (blockIdx.y ? A.dk_part : A.dq_part) + at / per_head * per_head * A.share +
                   at % per_head;
  f32x4 sum = *reinterpret_cast<const f32x4*>(p);
  for (int i = 1; i < A.share; ++i) sum += *reinterpret_cast<const f32x4*>(p + i * per_head);
  lin::Tile<T>::store4((T*)(blockIdx.y ? A.dk : A.dq) + at, sum);
}

template <class T>
hipError_t launch_share(const LinearArgs& a, int64_t per_head, hipStream_t stream) {
  const int64_t total = a.BH / a.share * per_head;
  hipLaunchKernelGGL((linear_share_kernel<T>),
                     dim3((unsigned)((total / 4 + kThreads - 1) / kThreads), 2), dim3(kThreads), 0,
                     stream, a, total, per_head);
  return hipGetLastError();
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t segment_bytes(int64_t BH, int nseg, int elems) {
  if (nseg == 1) return 0;
  return align256((size_t)BH * nseg * elems * 4) + align256((size_t)BH * nseg * 8);
}

void place_segments(LinearArgs& a, int elems, char*& ws) {
  if (a.nseg == 1) return;
  a.seg_state = (float*)ws;
  ws += align256((size_t)a.BH * a.nseg * elems * 4);
  a.seg_log = (double*)ws;
  ws += align256((size_t)a.BH * a.nseg * 8);
}

template <int kGroups, int kPer>
hipError_t launch_segments_by(const LinearArgs& a, int elems, bool reverse, hipStream_t stream) {
  const int64_t total = (int64_t)a.BH * elems;
  hipLaunchKernelGGL((linear_segments_kernel<kGroups, kPer>),
                     dim3((unsigned)(total / (4 * (kThreads / kGroups)))), dim3(kThreads), 0,
                     stream, a.seg_state, a.seg_log, a.S, total, elems, a.nseg, reverse);
  return hipGetLastError();
}

hipError_t launch_segments(const LinearArgs& a, int elems, bool reverse, hipStream_t stream) {
  if (a.nseg <= kOwnSegments) return hipSuccess;
  if (a.nseg <= 32) return launch_segments_by<8, 4>(a, elems, reverse, stream);
  return launch_segments_by<32, 16>(a, elems, reverse, stream);  // 512 at most
}

hipError_t launch_chunks(const LinearArgs& a, int dtype, int d_k, int d_v, int mode,
                         hipStream_t stream) {
  return dtype == 1 ? launch_linear_bf16(a, d_k, d_v, mode, stream)
                    : launch_linear_f32(a, d_k, d_v, mode, stream);
}

void set_segments(LinearArgs& a, int dtype, int elems, bool backward) {
  const int chunk = linear_chunk(dtype);
  a.nchunk = (int)((a.T + chunk - 1) / chunk);
  a.nseg = linear_segments(dtype, a.BH, a.T, elems, backward);
  a.seg_chunks = (a.nchunk + a.nseg - 1) / a.nseg;
  a.nseg = (a.nchunk + a.seg_chunks - 1) / a.seg_chunks;
}

// ---- one token of every memory: S = exp(g) S + k v^T, out = S^T q.  Bound by
// the state, read and written once: 1024 memories of 128 x 128 (134 MB) 20.5 us,
// 6.6 TB/s; one of 4 memories 2.4.  A workgroup takes all rows of CT columns, its
// loads in flight together: 64 of them (2048 memories of 64 x 64 11.3 us, by 32
// columns 12.7; 64 of 128 x 128 3.6 us, 3.4 by 32 columns and 4.1 by 128).
template <class T, int DK, int DV, int CT>
__global__ __launch_bounds__(kThreads) void linear_step_kernel(float* S, const T* q, const T* k,
                                                               const T* v, const float* g, T* out,
                                                               int share) {
  constexpr int kLanes = CT / 4;                 // lanes of a row piece
  constexpr int kRows = kThreads / kLanes;       // rows at a time
  constexpr int kN = DK / kRows;
  static_assert(DK % kRows == 0, "whole passes");
  __shared__ __align__(16) float sq[DK], sk[DK];
  __shared__ f32x4 sum[kThreads / kWave][kLanes];
  const int tid = threadIdx.x;
  const int64_t m = blockIdx.x / (DV / CT);
  const int c0 = (int)(blockIdx.x % (DV / CT)) * CT + (tid % kLanes) * 4;
  const int r0 = tid / kLanes;
  float* Sm = S + m * DK * DV + c0;
  f32x4 s[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i)
    s[i] = *reinterpret_cast<const f32x4*>(Sm + (r0 + i * kRows) * DV);
  const int64_t key = m / share * DK;
  if (tid < DK / 4) {
    const f32x4 a = lin::Tile<T>::load4(q + key + tid * 4);
    *reinterpret_cast<f32x4*>(sq + tid * 4) = a;
  } else if (tid >= kThreads - DK / 4) {
    const int i = tid - (kThreads - DK / 4);
    *reinterpret_cast<f32x4*>(sk + i * 4) = lin::Tile<T>::load4(k + key + i * 4);
  }
  const f32x4 vv = lin::Tile<T>::load4(v + m * DV + c0);
  const float a = expf(g[m]);
  __syncthreads();
  f32x4 o = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int r = r0 + i * kRows;
    s[i] = s[i] * a + vv * sk[r];
    *reinterpret_cast<f32x4*>(Sm + r * DV) = s[i];
    o += s[i] * sq[r];
  }
  // rows of the wavefront, then its sums in their order
#pragma unroll
  for (int x = kLanes; x < kWave; x <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], x);
  const int lane = lane_id(), w = tid / kWave;
  if (lane < kLanes) sum[w][lane] = o;
  __syncthreads();
  if (tid < kLanes) {
    o = sum[0][tid];
#pragma unroll
    for (int i = 1; i < kThreads / kWave; ++i) o += sum[i][tid];
    lin::Tile<T>::store4(out + m * DV + c0, o);
  }
}

template <class T, int DK, int DV>
hipError_t launch_step(float* S, int BH, int share, const void* q, const void* k, const void* v,
                       const float* g, void* out, hipStream_t stream) {
  constexpr int CT = DV < 64 ? DV : 64;
  hipLaunchKernelGGL((linear_step_kernel<T, DK, DV, CT>), dim3((unsigned)BH * (DV / CT)),
                     dim3(kThreads), 0, stream, S, (const T*)q, (const T*)k, (const T*)v, g,
                     (T*)out, share);
  return hipGetLastError();
}

template <class T>
hipError_t launch_step_type(float* S, int BH, int share, int d_k, int d_v, const void* q,
                            const void* k, const void* v, const float* g, void* out,
                            hipStream_t s) {
  switch (d_k * 1000 + d_v) {
    case 32032: return launch_step<T, 32, 32>(S, BH, share, q, k, v, g, out, s);
    case 32064: return launch_step<T, 32, 64>(S, BH, share, q, k, v, g, out, s);
    case 32128: return launch_step<T, 32, 128>(S, BH, share, q, k, v, g, out, s);
    case 64032: return launch_step<T, 64, 32>(S, BH, share, q, k, v, g, out, s);
    case 64064: return launch_step<T, 64, 64>(S, BH, share, q, k, v, g, out, s);
    case 64128: return launch_step<T, 64, 128>(S, BH, share, q, k, v, g, out, s);
    case 128032: return launch_step<T, 128, 32>(S, BH, share, q, k, v, g, out, s);
    case 128064: return launch_step<T, 128, 64>(S, BH, share, q, k, v, g, out, s);
    default: return launch_step<T, 128, 128>(S, BH, share, q, k, v, g, out, s);
  }
}

}  // namespace

// Segments of a memory's steps: as many as give every compute unit a workgroup
// (a chunk is a chain of dependent phases, 6 us forward and 18 back at 128 x 128
// in bf16, so chunks go side by side), two where a segment of at most 32 memories
// keeps 16 chunks even so (16 memories x 32768 steps, bf16: 225 us with two, 259
// with one; 32 of 64 x 128 x 2047 steps, fp32, the other way, 56 and 52, and 64 x
// 2048 with a tape 98 and 83).  Segments cost a kernel for their states and sums
// of these, 5 to 10 us.  Back they gain from 4 chunks on (4 memories x 250 steps of
// 128 x 128, bf16: 55 us in one piece, 32 cut; 64 x 256 58 and 40).  Forward a chunk
// takes 1.3 to 6 us.  Four segments or more gain from 5 chunks on (64 memories, in
// one piece and cut: 64 x 64 bf16 14.5 and 12.7 us, 64 x 128 19.6 and 17.3, 128 x 64
// 19.7 and 16.7, 128 x 128 26.8 and 23.9, fp32 33.9 and 27.7; 24 of 64 x 128
// 19.1 and 14.0), but by less than a launch takes on the host, 3.7 us, where heads
// are below 64 x 64 (64 memories of 64 x 32 12.6 and 11.0; from 8 chunks on 18.7 and
// 12.1).  Two segments (65 to 128 memories) gain from 8 on (128 of 64 x 128, 5
// chunks, 20.6 and 23.4; 8 chunks 30.3 and 30.3; of 64 x 32 18.8 and 17.7).
int linear_segments(int dtype, int64_t BH, int64_t T, int elems, bool backward) {
  const int64_t chunks = (T + linear_chunk(dtype) - 1) / linear_chunk(dtype);
  if (chunks < (backward ? 4 : elems >= 64 * 64 && BH <= 64 ? 5 : 8)) return 1;
  int64_t n = 256 / BH;
  if (!backward && BH <= 32 && chunks >= 16 * (512 / BH)) n = 512 / BH;
  if (n > chunks) n = chunks;
  return n < 1 ? 1 : (int)n;
}

size_t linear_scan_workspace_bytes(int dtype, int64_t BH, int d_k, int d_v, int64_t T) {
  return segment_bytes(BH, linear_segments(dtype, BH, T, d_k * d_v, false), d_k * d_v);
}

size_t linear_backward_workspace_bytes(int dtype, int64_t BH, int share, int d_k, int d_v,
                                       int64_t T) {
  const size_t part = share > 1 ? 2 * align256((size_t)BH * T * d_k * 4) : 0;
  return part + segment_bytes(BH, linear_segments(dtype, BH, T, d_k * d_v, true), d_k * d_v);
}

hipError_t launch_linear_scan(LinearArgs a, int dtype, int d_k, int d_v, void* ws,
                              hipStream_t stream) {
  set_segments(a, dtype, d_k * d_v, false);
  char* p = (char*)ws;
  place_segments(a, d_k * d_v, p);
  hipError_t rc;
  if (a.nseg > 1) {
    if ((rc = launch_chunks(a, dtype, d_k, d_v, 1, stream)) != hipSuccess) return rc;
    if ((rc = launch_segments(a, d_k * d_v, false, stream)) != hipSuccess) return rc;
  }
  return launch_chunks(a, dtype, d_k, d_v, 0, stream);
}

hipError_t launch_linear_backward(LinearArgs a, int dtype, int d_k, int d_v, void* ws,
                                  hipStream_t stream) {
  set_segments(a, dtype, d_k * d_v, true);
  char* p = (char*)ws;
  place_segments(a, d_k * d_v, p);
  const int64_t per_head = a.T * d_k;
  if (a.share > 1) {
    a.dq_part = (float*)p;
    p += align256((size_t)a.BH * per_head * 4);
    a.dk_part = (float*)p;
  }
  hipError_t rc;
  if (a.nseg > 1) {
    if ((rc = launch_chunks(a, dtype, d_k, d_v, 2, stream)) != hipSuccess) return rc;
    if ((rc = launch_segments(a, d_k * d_v, true, stream)) != hipSuccess) return rc;
  }
  rc = dtype == 1 ? launch_linear_backward_bf16(a, d_k, d_v, stream)
                  : launch_linear_backward_f32(a, d_k, d_v, stream);
  if (rc != hipSuccess || a.share == 1) return rc;
  return dtype == 1 ? launch_share<uint16_t>(a, per_head, stream)
                    : launch_share<float>(a, per_head, stream);
}

hipError_t launch_linear_step(float* S, int dtype, int BH, int share, int d_k, int d_v,
                              const void* q, const void* k, const void* v, const float* g,
                              void* out, hipStream_t stream) {
  return dtype == 1
             ? launch_step_type<uint16_t>(S, BH, share, d_k, d_v, q, k, v, g, out, stream)
             : launch_step_type<float>(S, BH, share, d_k, d_v, q, k, v, g, out, stream);
}

}  // namespace sdm
