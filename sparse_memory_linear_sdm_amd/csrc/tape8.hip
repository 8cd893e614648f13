// Reading the 8-bit tape back (mx.h, 8-bit form): codes [n_mem, d_v/16, S, 16]
// and scale bytes [n_mem, d_v/16, S], S = T * (W + R) row records, to rows
// [n_mem, S, d_v] in fp32 or bf16 (exact in both).  A stream bound by memory.
// A thread turns one record (16 code bytes, a scale) into a row's 16 columns;
// the d_v/16 threads of a row are neighbours.  In bf16 a record is two 16-byte
// pieces of the output: lanes 2m and 2m + 1 take records m and m + 32 of the
// wavefront's 64 and swap halves, so that each of its two stores is 1 KiB in a
// row and can pass the caches.  In fp32 it is four, and the lanes of a quad take
// records 16 apart and exchange pieces, to the same end.  64 memories x 512
// steps of 128 rows of 128 values: 475 us in fp32 (5.7 TB/s; 663 with a lane's
// pieces stored as they lie), 300 us in bf16.
#include "internal.h"
#include "mx.h"

namespace sdm {
namespace {

template <typename T, typename I>
__global__ __launch_bounds__(256) void tape8_read_kernel(const u32x4* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t S, int lognb, int64_t records,
                                                         u32x4* __restrict__ rows) {
  const I n = (I)records, s_rows = (I)S, step = (I)gridDim.x * 256;
  const int lane = lane_id();
  // whole wavefronts: the lanes past the end only take part in the exchange
  for (I i0 = (I)blockIdx.x * 256 + (threadIdx.x & ~63u); i0 < n; i0 += step) {
    const I i = i0 + (sizeof(T) == 2 ? (lane >> 1) + 32 * (lane & 1) : (lane >> 2) + 16 * (lane & 3));
    u32x4 c = {0u, 0u, 0u, 0u};
    uint32_t b = kMxMinScale;
    if (i < n) {
      const I row = i >> lognb, mem = row / s_rows;
      const int64_t rec = (((int64_t)mem << lognb) + (int64_t)(i & (((I)1 << lognb) - 1))) * S +
                          (int64_t)(row - mem * s_rows);
      c = codes[rec];
      b = scales[rec];
    }
    const float s = scale_value(b);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t f[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[4];
      int8_unpack4(w[k], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[4 * k + j] = __float_as_uint(x[j] * s);
    }
    if constexpr (sizeof(T) == 2) {
      const bool odd = lane & 1;
      uint32_t lo[4], hi[4];  // the wavefront's pieces 0..63 and 64..127
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // seven significant bits: the upper halves are exact
        const uint32_t h0 = (f[2 * k] >> 16) | (f[2 * k + 1] & 0xFFFF0000u);
        const uint32_t h1 = (f[8 + 2 * k] >> 16) | (f[8 + 2 * k + 1] & 0xFFFF0000u);
        const uint32_t got = dpp_mov<0xB1>(odd ? h0 : h1);
        lo[k] = odd ? got : h0;
        hi[k] = odd ? h1 : got;
      }
      const I p = 2 * i0 + lane;
      if (p < 2 * n) __builtin_nontemporal_store(u32x4{lo[0], lo[1], lo[2], lo[3]}, rows + p);
      if (p + 64 < 2 * n)
        __builtin_nontemporal_store(u32x4{hi[0], hi[1], hi[2], hi[3]}, rows + p + 64);
    } else {
      uint32_t g[4][4];  // word e of piece j of the lane's record; then of record j's piece lane % 4
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) g[e][j] = f[4 * j + e];
        quad_transpose(g[e]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // records i0 + 16 j .. + 15
        const I p = 4 * i0 + 64 * j + lane;
        if (p < 4 * n)
          __builtin_nontemporal_store(u32x4{g[0][j], g[1][j], g[2][j], g[3][j]}, rows + p);
      }
    }
  }
}

template <typename T>
void launch_read(const int8_t* tape, const uint8_t* tape_scale, int n_mem, int d_v, int64_t S,
                 void* rows, hipStream_t stream) {
  int lognb = 0;
  while ((16 << lognb) < d_v) ++lognb;  // d_v is 16 times a power of two
  const int64_t n = ((int64_t)n_mem * S) << lognb;
  int64_t blocks = (n + 255) / 256;
  if (blocks > kMaxStrideBlocks) blocks = kMaxStrideBlocks;  // the loop strides over the rest
  const u32x4* const c = reinterpret_cast<const u32x4*>(tape);
  u32x4* const o = reinterpret_cast<u32x4*>(rows);
  if (n <= ((int64_t)1 << 29))  // four pieces a record: every index stays below 2^32
    hipLaunchKernelGGL((tape8_read_kernel<T, uint32_t>), dim3((unsigned)blocks), dim3(256), 0,
                       stream, c, tape_scale, S, lognb, n, o);
  else
    hipLaunchKernelGGL((tape8_read_kernel<T, uint64_t>), dim3((unsigned)blocks), dim3(256), 0,
                       stream, c, tape_scale, S, lognb, n, o);
}

}  // namespace

hipError_t launch_tape8_read(const int8_t* tape, const uint8_t* tape_scale, int dtype, int n_mem,
                             int d_v, int64_t S, void* rows, hipStream_t stream) {
  if (S == 0) return hipSuccess;
  if (dtype == 1)
    launch_read<uint16_t>(tape, tape_scale, n_mem, d_v, S, rows, stream);
  else
    launch_read<float>(tape, tape_scale, n_mem, d_v, S, rows, stream);
  return hipGetLastError();
}

}  // namespace sdm
