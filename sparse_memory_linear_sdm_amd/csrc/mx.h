// Microscaled formats: blocks of consecutive values that share one scale, a
// power of two held as its biased exponent in a byte (code b stands for
// 2^(b - 127); 255 marks a block that holds a NaN or an infinity, all of whose
// values read as NaN).  Two of them:
//   4-bit   blocks of 32, elements e2m1 (sign, 2 exponent bits, 1 mantissa
//           bit: 0, .5, 1, 1.5, 2, 3, 4, 6); scale 2^(floor(log2 max|x|) - 2),
//           so that the largest value lands in [4, 8) and rounds to 4 or 6
//           (larger ones are held at 6);
//   8-bit   blocks of 16, elements two's complement integers in [-127, 127];
//           the smallest scale that keeps the rounded codes in that range.
// Scales stop at 2^-125 (code 2), so that every value is a normal binary32
// number or zero; smaller blocks round towards zero on that grid.
#pragma once
#include "device_common.h"

namespace sdm {

constexpr uint32_t kMxMinScale = 2;
constexpr uint32_t kMxNan = 255;
constexpr uint32_t kF32Inf = 0x7F800000u;  // binary32 magnitudes from here on are not finite

// Magnitude bits of a binary32 value: they order like the magnitudes, and a
// NaN counts above infinity, so a block's maximum of them also finds both.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest of four values' magnitude bits (the maximum that a NaN wins).
__device__ __forceinline__ uint32_t max_mag4(const u32x4& x) {
  const float a = __builtin_elementwise_maximum(fabsf(__uint_as_float(x.x)), fabsf(__uint_as_float(x.y)));
  const float b = __builtin_elementwise_maximum(a, fabsf(__uint_as_float(x.z)));
  return mag_bits(__builtin_elementwise_maximum(b, fabsf(__uint_as_float(x.w))));
}

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = umax(m, dpp_qp_xor1(m));
  return umax(m, dpp_qp_xor2(m));
}

// 2^(b - 127) for b in [1, 254].
__device__ __forceinline__ float scale_f32(uint32_t b) { return __uint_as_float(b << 23); }

// What any scale code stands for: 2^(b - 127), for 0 a subnormal; NaN for 255,
// whose bits are infinity's and the product with zero NaN.
__device__ __forceinline__ float scale_value(uint32_t b) {
  const float s = __uint_as_float(umax(b << 23, 0x00400000u));
  return fmaf(s, 0.0f, s);
}

// Scale code of a 4-bit block from its maximum's magnitude bits.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t m) {
  const int e = (int)(m >> 23) - 2;
  return m >= kF32Inf ? kMxNan : (e < (int)kMxMinScale ? kMxMinScale : (uint32_t)e);
}

// Scale code of an 8-bit block: 2^(floor(log2 m) - 6), doubled where m would
// round to 128, i.e. from 127.5 scales on -- exactly where the mantissa's top
// seven bits are all set, so adding one there carries into the exponent.
__device__ __forceinline__ uint32_t int8_scale(uint32_t m) {
  const int e = (int)((m + 0x10000u) >> 23) - 6;
  return m >= kF32Inf ? kMxNan : (e < (int)kMxMinScale ? kMxMinScale : (uint32_t)e);
}

// Bits of the inverse scale 2^(127 - b).
__device__ __forceinline__ uint32_t int8_inverse(uint32_t b) { return (254u - b) << 23; }

// Four values (binary32 bits) times the inverse scale of their block, rounded
// to nearest even, as two's complement bytes.  The product is exact and at
// most 127.5 in magnitude, so adding 1.5 * 2^23 leaves the rounded integer in
// the low byte of the sum.  (Of no meaning in a block marked 255.)
__device__ __forceinline__ uint32_t int8_pack4(const u32x4& x, float inv) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t q0 = __float_as_uint(fmaf(__uint_as_float(x.x), inv, kMagic));
  const uint32_t q1 = __float_as_uint(fmaf(__uint_as_float(x.y), inv, kMagic));
  const uint32_t q2 = __float_as_uint(fmaf(__uint_as_float(x.z), inv, kMagic));
  const uint32_t q3 = __float_as_uint(fmaf(__uint_as_float(x.w), inv, kMagic));
  const uint32_t lo = __builtin_amdgcn_perm(q1, q0, 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(q3, q2, 0x04000C0Cu);
  return lo | hi;
}

// The four integers of a code word as binary32 (exact).
__device__ __forceinline__ void int8_unpack4(uint32_t w, float (&x)[4]) {
  const uint32_t u = w ^ 0x80808080u;  // offset binary: the unsigned byte conversions apply
  x[0] = (float)(u & 0xFFu) - 128.0f;
  x[1] = (float)((u >> 8) & 0xFFu) - 128.0f;
  x[2] = (float)((u >> 16) & 0xFFu) - 128.0f;
  x[3] = (float)(u >> 24) - 128.0f;
}

// 4 x 4 transpose across the lanes of a quad: lane p's word k goes to word p
// of lane k.  Two exchange steps (lanes 1 apart, then 2), each swapping the
// off-diagonal words of a 2 x 2 block of (lanes, words).
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4]) {
  const int lane = lane_id();
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t got = dpp_mov<0xB1>(odd ? w[i] : w[i + 1]);
    w[i] = odd ? got : w[i];
    w[i + 1] = odd ? w[i + 1] : got;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t got = dpp_mov<0x4E>(high ? w[i] : w[i + 2]);
    w[i] = high ? got : w[i];
    w[i + 2] = high ? w[i + 2] : got;
  }
}

}  // namespace sdm
