// 4-bit microscaled matrices (mx.h): quantisation of fp32 or bf16 rows and
// reading them back.
//
// Layout.  codes [rows, cols/2] bytes, the even column in the low nibble;
// scales [cols/128, rows, 4] bytes: byte j of entry (g, r) is the scale of
// columns 128 g + 32 j .. + 31 of row r.  The scales of one 128-column group
// lie together for consecutive rows, as the product's tiles load them (one
// 4-byte word per row and 128 columns).
//
// Both passes are streams bound by memory: each value is read once and
// written once.  A workgroup takes a tile of kQuantRows rows; tiles follow each
// other along the columns, so that the chip walks whole rows of the matrix
// (down the rows first: 326 against 216 us for 32768 x 16384 bf16; 4 and 16
// rows a tile: 219 and 235).  Quantisation: a wavefront reads 512 columns of a
// row at a time (8 values per lane: one 16-byte load of bf16, two of fp32), the
// block maximum is two exchanges over the four lanes that share a block, and
// the scale words are gathered in LDS so that the rows' words of each group go
// out together.  32768 x 16384 bf16: 216-228 us (6.0-6.3 TB/s) and
// 216-233 us back; 4226 x 16384 fp32: 47-50 and 44 us.
#include "internal.h"
#include "mx.h"

namespace sdm {
namespace {

constexpr int kQCols = 512;  // columns of a workgroup's tile: 8 per lane
constexpr int kQWaves = 4;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const u32x4 q = *reinterpret_cast<const u32x4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 q = reinterpret_cast<const f32x4*>(p)[i];
      x[4 * i] = q.x;
      x[4 * i + 1] = q.y;
      x[4 * i + 2] = q.z;
      x[4 * i + 3] = q.w;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kQWaves* kWave) void quantize_kernel(const T* __restrict__ x,
                                                                  int64_t rows, int cols,
                                                                  uint32_t* __restrict__ codes,
                                                                  uint32_t* __restrict__ scales) {
  __shared__ uint32_t sc[kQCols / 128][kQuantRows];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const uint32_t tiles = (uint32_t)(cols + kQCols - 1) / kQCols, rowtile = blockIdx.x / tiles;
  const int64_t r0 = (int64_t)rowtile * kQuantRows;
  const int c0 = (int)(blockIdx.x - rowtile * tiles) * kQCols, c = c0 + lane * 8;
  constexpr int kEach = kQuantRows / kQWaves;
  float v[kEach][8];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t r = r0 + wave * kEach + i;
    if (r < rows && c < cols) {
      load8(x + r * cols + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t r = r0 + wave * kEach + i;
    float top = 0.0f;  // the maximum that a NaN wins
#pragma unroll
    for (int j = 0; j < 8; ++j) top = __builtin_elementwise_maximum(top, fabsf(v[i][j]));
    const uint32_t b = mx4_scale(quad_max(mag_bits(top)));  // a block of 32 is four lanes of 8
    const float s = scale_f32(b);
    uint32_t q = 0;  // the conversion divides by s, rounds to nearest even and holds at +-6
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[i][0], v[i][1], s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[i][2], v[i][3], s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[i][4], v[i][5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[i][6], v[i][7], s, 3);
    if (r < rows && c < cols) codes[(r * cols + c) / 8] = b == kMxNan ? 0u : q;
    if ((lane & 3) == 0)
      reinterpret_cast<uint8_t*>(&sc[lane / 16][wave * kEach + i])[(lane / 4) & 3] = (uint8_t)b;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kQCols / 128 * kQuantRows; i += kQWaves * kWave) {
    const int g = c0 / 128 + i / kQuantRows;
    const int64_t r = r0 + i % kQuantRows;
    if (g < cols / 128 && r < rows) scales[(int64_t)g * rows + r] = sc[i / kQuantRows][i % kQuantRows];
  }
}

// Reading back: a thread takes 16 bytes of output (8 bf16 values from a word of
// codes, 4 fp32 values from half a word) in each of its wavefront's rows, so
// that the stores are contiguous.
template <typename T>
__global__ __launch_bounds__(kQWaves* kWave) void dequantize_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int cols,
    u32x4* __restrict__ x) {
  constexpr int kEach = 16 / sizeof(T), kCols = kWave * kEach, kRows = kQuantRows / kQWaves;
  static_assert(kCols == dequantize_cols(sizeof(T)), "the host's count of tiles");
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const uint32_t tiles = (uint32_t)(cols + kCols - 1) / kCols, rowtile = blockIdx.x / tiles;
  const int c = (int)(blockIdx.x - rowtile * tiles) * kCols + lane * kEach;
  if (c >= cols) return;
  const int64_t r0 = (int64_t)rowtile * kQuantRows + wave * kRows;
  uint32_t q[kRows], b[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + i < rows ? r0 + i : rows - 1;
    if constexpr (kEach == 8)
      q[i] = reinterpret_cast<const uint32_t*>(codes)[(r * cols + c) / kEach];
    else
      q[i] = reinterpret_cast<const uint16_t*>(codes)[(r * cols + c) / kEach];
    b[i] = scales[((int64_t)(c / 128) * rows + r) * 4 + (c / 32) % 4];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (r0 + i >= rows) return;
    const float s = scale_value(b[i]);
    float f[kEach];
    const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 0);
    const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[j] = p0[j] * s;
      f[2 + j] = p1[j] * s;
    }
    u32x4 o;
    if constexpr (kEach == 8) {
      const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 2);
      const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 3);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f[4 + j] = p2[j] * s;
        f[6 + j] = p3[j] * s;
      }
      // two significant bits down to 2^-128: exact in bf16, by the upper halves
      o.x = (__float_as_uint(f[0]) >> 16) | (__float_as_uint(f[1]) & 0xFFFF0000u);
      o.y = (__float_as_uint(f[2]) >> 16) | (__float_as_uint(f[3]) & 0xFFFF0000u);
      o.z = (__float_as_uint(f[4]) >> 16) | (__float_as_uint(f[5]) & 0xFFFF0000u);
      o.w = (__float_as_uint(f[6]) >> 16) | (__float_as_uint(f[7]) & 0xFFFF0000u);
    } else {
      o = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                __float_as_uint(f[3])};
    }
    // a stream, past the caches: 44 against 58 us for 4226 x 16384 fp32
    __builtin_nontemporal_store(o, x + ((r0 + i) * cols + c) / kEach);
  }
}

template <typename T>
hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols,
                             void* x, hipStream_t stream) {
  const int64_t blocks = dequantize_blocks(rows, cols, sizeof(T));
  hipLaunchKernelGGL((dequantize_kernel<T>), dim3((unsigned)blocks), dim3(kQWaves * kWave), 0,
                     stream, codes, scales, rows, cols, reinterpret_cast<u32x4*>(x));
  return hipGetLastError();
}

template <typename T>
hipError_t launch_quantize(const void* x, int64_t rows, int cols, uint8_t* codes, uint8_t* scales,
                           hipStream_t stream) {
  hipLaunchKernelGGL((quantize_kernel<T>), dim3((unsigned)quantize_blocks(rows, cols)),
                     dim3(kQWaves * kWave), 0, stream, reinterpret_cast<const T*>(x), rows, cols,
                     reinterpret_cast<uint32_t*>(codes), reinterpret_cast<uint32_t*>(scales));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_quantize(const void* x, int dtype, int64_t rows, int cols, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream) {
  return dtype == 1 ? launch_quantize<uint16_t>(x, rows, cols, codes, scales, stream)
                    : launch_quantize<float>(x, rows, cols, codes, scales, stream);
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype,
                                 int64_t rows, int cols, void* x, hipStream_t stream) {
  return dtype == 1 ? launch_dequantize<uint16_t>(codes, scales, rows, cols, x, stream)
                    : launch_dequantize<float>(codes, scales, rows, cols, x, stream);
}

}  // namespace sdm
