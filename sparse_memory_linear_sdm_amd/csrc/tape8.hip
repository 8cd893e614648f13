// Reading the 8-bit tape back (mx.h, 8-bit form): codes [n_mem, d_v/16, S, 16]
// and scale bytes [n_mem, d_v/16, S], S = T * (W + R) row records, to rows
// [n_mem, S, d_v] in fp32 or bf16 (exact in both).  A stream bound by memory;
// each thread turns one record (16 code bytes) into a row's 16 columns.  The
// d_v/16 threads of a row are neighbours, so a wavefront writes whole rows
// and reads runs of 64 / (d_v/16) records from each block.
#include "internal.h"
#include "mx.h"

namespace sdm {
namespace {

template <typename T>
__global__ __launch_bounds__(256) void tape8_read_kernel(const u32x4* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t S, int lognb, int64_t n,
                                                         u32x4* __restrict__ rows) {
  const int nb = 1 << lognb;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i >> lognb, mem = row / S;
    const int64_t rec = ((mem << lognb) + (i & (nb - 1))) * S + (row - mem * S);
    const u32x4 c = codes[rec];
    const uint32_t b = scales[rec];
    const float s = b == kMxNan ? __uint_as_float(0x7FC00000u)
                                : (b == 0 ? __uint_as_float(0x00400000u) : scale_f32(b));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t f[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[4];
      int8_unpack4(w[k], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[4 * k + j] = __float_as_uint(x[j] * s);
    }
    if constexpr (sizeof(T) == 2) {  // seven significant bits: the upper halves are exact
#pragma unroll
      for (int k = 0; k < 2; ++k)
        rows[2 * i + k] = u32x4{(f[8 * k] >> 16) | (f[8 * k + 1] & 0xFFFF0000u),
                                (f[8 * k + 2] >> 16) | (f[8 * k + 3] & 0xFFFF0000u),
                                (f[8 * k + 4] >> 16) | (f[8 * k + 5] & 0xFFFF0000u),
                                (f[8 * k + 6] >> 16) | (f[8 * k + 7] & 0xFFFF0000u)};
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        rows[4 * i + k] = u32x4{f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]};
    }
  }
}

}  // namespace

hipError_t launch_tape8_read(const int8_t* tape, const uint8_t* tape_scale, int dtype, int n_mem,
                             int d_v, int64_t S, void* rows, hipStream_t stream) {
  int lognb = 0;
  while ((16 << lognb) < d_v) ++lognb;  // d_v is 16 times a power of two
  const int64_t n = ((int64_t)n_mem * S) << lognb;
  if (n == 0) return hipSuccess;
  int64_t blocks = (n + 255) / 256;
  if (blocks > kMaxStrideBlocks) blocks = kMaxStrideBlocks;  // the loop strides over the rest
  const u32x4* const c = reinterpret_cast<const u32x4*>(tape);
  u32x4* const o = reinterpret_cast<u32x4*>(rows);
  if (dtype == 1)
    hipLaunchKernelGGL(tape8_read_kernel<uint16_t>, dim3((unsigned)blocks), dim3(256), 0, stream,
                       c, tape_scale, S, lognb, n, o);
  else
    hipLaunchKernelGGL(tape8_read_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, stream, c,
                       tape_scale, S, lognb, n, o);
  return hipGetLastError();
}

}  // namespace sdm
