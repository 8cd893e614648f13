// Matrix-core tiles of the dense recurrence: fragments of 16 x 32 and
// 32 x 16 operands for 16 x 16 products, in bf16 or fp32.
//
// Every product runs over 32 values of its inner index at a time.  Lane l of
// the wavefront (g = l / 16) holds, for row or column l % 16 of the operand,
// the inner values 16 * (j / 4) + 4 g + j % 4, j = 0..7.  An accumulator tile
// (row 4 g + i, column l % 16, i = 0..3) holds its rows in the same order, so
// two accumulator tiles one below the other are an operand of the next product
// as they stand, whose inner index is their row.  (The instructions' own order
// of the inner index does not matter while both operands agree.)
//   bf16  one v_mfma_f32_16x16x32_bf16;
//   fp32  eight v_mfma_f32_16x16x4_f32, the j-th values of each.
#pragma once
#include "device_common.h"

namespace sdm {
namespace lin {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// LDS rows are padded by 16 bytes: rows start 4 banks apart (of 64), so that
// both kinds of fragment reads spread evenly over the banks.
template <class T>
struct Tile;

template <>
struct Tile<uint16_t> {
  static constexpr int kChunk = 64;  // steps
  static constexpr int kPad = 8;     // values
  // Parts of a scaled operand whose product must keep fp32's precision: a bf16
  // part holds 8 of the 24 bits.
  static constexpr int kParts = 3;
  typedef bf16x8 Frag;

  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // Row `row0 + l % 16` of an LDS matrix, inner values k0 .. k0 + 31 along it.
  static __device__ __forceinline__ Frag rows(const uint16_t* m, int ld, int row0, int k0) {
    const int l = lane_id();
    const uint16_t* p = m + (row0 + (l & 15)) * ld + k0 + 4 * (l >> 4);
    const bf16x4 a = *reinterpret_cast<const bf16x4*>(p);
    const bf16x4 b = *reinterpret_cast<const bf16x4*>(p + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  // Column `col0 + l % 16`, inner values k0 .. k0 + 31 down the rows: transposed
  // reads (16 lanes read 4 rows of 16 values, each gets one column).
  static __device__ __forceinline__ Frag cols(const uint16_t* m, int ld, int k0, int col0) {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const int l = lane_id();
    const uint16_t* p = m + (k0 + 4 * (l >> 4) + ((l & 15) >> 2)) * ld + col0 + 4 * (l & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 16 * ld));
    return __builtin_shufflevector(__builtin_bit_cast(bf16x4, a), __builtin_bit_cast(bf16x4, b),
                                   0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ Frag pack(f32x4 a, f32x4 b) {
    return __builtin_shufflevector(__builtin_convertvector(a, bf16x4),
                                   __builtin_convertvector(b, bf16x4), 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ f32x8 widen(Frag a) {
    return __builtin_convertvector(a, f32x8);
  }
  // x as the sum of kParts operands, to within 2^-26 of it
  static __device__ __forceinline__ void split(f32x8 x, Frag* part) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      part[p] = __builtin_convertvector(x, bf16x8);
      x = x - __builtin_convertvector(part[p], f32x8);
    }
  }
  static __device__ __forceinline__ void store4(uint16_t* p, f32x4 x) {
    *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(x, bf16x4);
  }
  static __device__ __forceinline__ f32x4 load4(const uint16_t* p) {
    return __builtin_convertvector(*reinterpret_cast<const bf16x4*>(p), f32x4);
  }
};

template <>
struct Tile<float> {
  static constexpr int kChunk = 32;
  static constexpr int kPad = 4;
  static constexpr int kParts = 1;
  typedef f32x8 Frag;

  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Frag rows(const float* m, int ld, int row0, int k0) {
    const int l = lane_id();
    const float* p = m + (row0 + (l & 15)) * ld + k0 + 4 * (l >> 4);
    return pack(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 16));
  }
  static __device__ __forceinline__ Frag cols(const float* m, int ld, int k0, int col0) {
    const int l = lane_id();
    const float* p = m + (k0 + 4 * (l >> 4)) * ld + col0 + (l & 15);
    Frag f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = p[(16 * (j / 4) + j % 4) * ld];
    return f;
  }
  static __device__ __forceinline__ Frag pack(f32x4 a, f32x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ f32x8 widen(Frag a) { return a; }
  static __device__ __forceinline__ void split(f32x8 x, Frag* part) { part[0] = x; }
  static __device__ __forceinline__ void store4(float* p, f32x4 x) {
    *reinterpret_cast<f32x4*>(p) = x;
  }
  static __device__ __forceinline__ f32x4 load4(const float* p) {
    return *reinterpret_cast<const f32x4*>(p);
  }
};

// One [kChunk, D] block of a [T, D] array: 16-byte pieces through registers
// into LDS rows of D + kPad values, zeros behind the last step.
template <class T, int D, int THREADS>
struct Block {
  static constexpr int kC = Tile<T>::kChunk;
  static constexpr int kLd = D + Tile<T>::kPad;
  static constexpr int kRowPieces = D * (int)sizeof(T) / 16;
  static constexpr int kPieces = kC * kRowPieces;
  static constexpr int kN = (kPieces + THREADS - 1) / THREADS;
  u32x4 r[kN];

  __device__ __forceinline__ void load(const T* base, int valid_rows) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int p = threadIdx.x + i * THREADS;
      r[i] = u32x4{0, 0, 0, 0};
      if (p < kPieces && p / kRowPieces < valid_rows)
        r[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(base) + p * 16);
    }
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int p = threadIdx.x + i * THREADS;
      if (p < kPieces)
        *reinterpret_cast<u32x4*>(lds + (p / kRowPieces) * kLd +
                                  (p % kRowPieces) * (16 / (int)sizeof(T))) = r[i];
    }
  }
};

// Decays of one chunk.  The sums of logarithms are formed in 64 bits and kept
// as two floats, so that the decay between two steps has fp32's precision
// whatever other steps of the chunk forget.
template <int C>
struct Decays {
  float hi[C], lo[C];  // log2 of the decay from the chunk's start through step t
  float into[C];       // that decay
  float onto[C];       // decay behind step t to the chunk's end
  float whole;         // of the whole chunk
};

// log2 of one step's decay.  Below 2^-184 = exp(-128) it is 0 in fp32 with
// any number of further steps; so is -infinity's, without infinities here.
__device__ __forceinline__ double log2_decay(float g) {
  return (double)(g < -128.0f ? -128.0f : g) * 1.4426950408889634;
}

// By one whole wavefront, step `lane`'s x (0 behind the last step and in lanes
// at or past C): fills d and returns the chunk's sum.
template <int C>
__device__ __forceinline__ double scan_decays(double x, Decays<C>& d) {
  const int l = lane_id();
#pragma unroll
  for (int o = 1; o < C; o <<= 1) {
    const double y = __shfl_up(x, o);
    if (l >= o) x += y;
  }
  const double sum = __shfl(x, C - 1);
  if (l < C) {
    const float hi = (float)x;
    d.hi[l] = hi;
    d.lo[l] = (float)(x - (double)hi);
    d.into[l] = exp2f(hi);
    d.onto[l] = exp2f((float)(sum - x));
    if (l == 0) d.whole = exp2f((float)sum);
  }
  return sum;
}

// decay behind step s through step t >= s
template <int C>
__device__ __forceinline__ float decay_between(const Decays<C>& d, int t, int s) {
  return exp2f((d.hi[t] - d.hi[s]) + (d.lo[t] - d.lo[s]));
}

// A contiguous range of memories per XCD (workgroups go to the 8 XCDs in turn),
// so that heads that share keys share an L2.
__device__ __forceinline__ int64_t xcd_contiguous(int64_t block, int64_t n) {
  return n % 8 == 0 ? (block & 7) * (n / 8) + (block >> 3) : block;
}

}  // namespace lin
}  // namespace sdm
