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

// LDS matrices of rows of D values, padded by 16 bytes: rows start 4 banks apart
// (of 64), so that reads along rows and fp32's along columns touch every bank
// once, at addresses with constant distances.  (bf16's transposed reads meet
// twice in a bank.  16-byte segments that change places by the row avoid that
// and cost more in address arithmetic and in register moves.)
template <class T>
struct Tile;

template <>
struct Tile<uint16_t> {
  static constexpr int kChunk = 64;  // steps
  template <int D>
  static constexpr int kLd = D + 8;  // values from row to row
  template <int D>
  static __device__ __forceinline__ int at(int row, int col) {
    return row * kLd<D> + col;
  }
  // Parts of a scaled operand whose product must keep fp32's precision: a bf16
  // part holds 8 of the 24 bits.
  static constexpr int kParts = 3;
  // Parts of what fp32 holds (the state, products of steps) where a sum is rounded
  // to bf16 behind the product: two are off by 2^-16 of it at most, beside the 2^-8
  // of the rounding.  (One part, 2^-8 of every term, puts outputs 1.4 times as far
  // from the exact ones as the rounding alone.)
  static constexpr int kOutParts = 2;
  static constexpr int kRowReads = 1, kColReads = 2, kProducts = 1;  // instructions
  typedef bf16x8 Frag;

  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // Row `row0 + l % 16` of an LDS matrix, inner values k0 .. k0 + 31 along it.
  template <int D>
  static __device__ __forceinline__ Frag rows(const uint16_t* m, int row0, int k0) {
    const int l = lane_id();
    const uint16_t* p = m + at<D>(row0 + (l & 15), k0 + 4 * (l >> 4));
    const bf16x4 a = *reinterpret_cast<const bf16x4*>(p);
    const bf16x4 b = *reinterpret_cast<const bf16x4*>(p + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  // Column `col0 + l % 16`, inner values k0 .. k0 + 31 down the rows: transposed
  // reads (16 lanes read 4 rows of 16 values, each gets one column).
  template <int D>
  static __device__ __forceinline__ Frag cols(const uint16_t* m, int k0, int col0) {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const int l = lane_id();
    const uint16_t* p = m + at<D>(k0 + 4 * (l >> 4) + ((l & 15) >> 2), col0 + 4 * (l & 3));
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 16 * kLd<D>));
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
  // x as the sum of N operands, to within 2^-8N of it
  template <int N = kParts>
  static __device__ __forceinline__ void split(f32x8 x, Frag* part) {
#pragma unroll
    for (int p = 0; p < N; ++p) {
      part[p] = __builtin_convertvector(x, bf16x8);
      x = x - __builtin_convertvector(part[p], f32x8);
    }
  }
  // x stored as the sum of kOutParts matrices, `size` values apart
  static __device__ __forceinline__ void store4_parts(uint16_t* p, int size, f32x4 x) {
#pragma unroll
    for (int i = 0; i < kOutParts; ++i) {
      const bf16x4 part = __builtin_convertvector(x, bf16x4);
      *reinterpret_cast<bf16x4*>(p + i * size) = part;
      x = x - __builtin_convertvector(part, f32x4);
    }
  }
  static __device__ __forceinline__ void store4(uint16_t* p, f32x4 x) {
    *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(x, bf16x4);
  }
  static __device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t b, int at, f32x4 x) {
    __builtin_amdgcn_raw_buffer_store_b64(
        __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4)), b, at * 2, 0, 0);
  }
  static __device__ __forceinline__ f32x4 load4(const uint16_t* p) {
    return __builtin_convertvector(*reinterpret_cast<const bf16x4*>(p), f32x4);
  }
};

template <>
struct Tile<float> {
  static constexpr int kChunk = 32;
  template <int D>
  static constexpr int kLd = D + 4;
  template <int D>
  static __device__ __forceinline__ int at(int row, int col) {
    return row * kLd<D> + col;
  }
  static constexpr int kParts = 1, kOutParts = 1;
  static constexpr int kRowReads = 2, kColReads = 8, kProducts = 8;
  typedef f32x8 Frag;

  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
  template <int D>
  static __device__ __forceinline__ Frag rows(const float* m, int row0, int k0) {
    const int l = lane_id();
    const float* p = m + at<D>(row0 + (l & 15), k0 + 4 * (l >> 4));
    return pack(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 16));
  }
  template <int D>
  static __device__ __forceinline__ Frag cols(const float* m, int k0, int col0) {
    const int l = lane_id();
    const float* p = m + at<D>(k0 + 4 * (l >> 4), col0 + (l & 15));
    Frag f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = p[(16 * (j / 4) + j % 4) * kLd<D>];
    return f;
  }
  static __device__ __forceinline__ Frag pack(f32x4 a, f32x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ f32x8 widen(Frag a) { return a; }
  template <int N = kParts>
  static __device__ __forceinline__ void split(f32x8 x, Frag* part) {
    part[0] = x;
  }
  static __device__ __forceinline__ void store4_parts(float* p, int, f32x4 x) {
    *reinterpret_cast<f32x4*>(p) = x;
  }
  static __device__ __forceinline__ void store4(float* p, f32x4 x) {
    *reinterpret_cast<f32x4*>(p) = x;
  }
  static __device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t b, int at, f32x4 x) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b, at * 4, 0, 0);
  }
  static __device__ __forceinline__ f32x4 load4(const float* p) {
    return *reinterpret_cast<const f32x4*>(p);
  }
};

// A matrix of pairs of a chunk's steps (t, s), s <= t, in LDS: rows t below 32
// have columns for s below 32 only (with two parts of it the padded square of 64 x
// 64 would leave reverse passes of 64 x 64 heads one workgroup a compute unit).
template <class T>
struct Pairs {
  typedef Tile<T> X;
  static constexpr int kUpper = 32 * X::template kLd<32>;
  static constexpr int kSize = kUpper + (X::kChunk == 64 ? 32 * X::template kLd<64> : 0);
  static constexpr int kParts = X::kOutParts;
  static __device__ __forceinline__ void store4(T* m, int t, int s, f32x4 x) {  // four s
    X::store4_parts(m + (t < 32 ? X::template at<32>(t, s) : kUpper + X::template at<64>(t - 32, s)),
                    kSize, x);
  }
  // Step t0 + l % 16, inner values s0 .. s0 + 31.
  static __device__ __forceinline__ typename X::Frag rows(const T* m, int part, int t0, int s0) {
    m += part * kSize;
    return t0 < 32 ? X::template rows<32>(m, t0, s0) : X::template rows<64>(m + kUpper, t0 - 32, s0);
  }
  // Step s0 + l % 16, inner values t0 .. t0 + 31 (t0 a multiple of 32).
  static __device__ __forceinline__ typename X::Frag cols(const T* m, int part, int t0, int s0) {
    m += part * kSize;
    return t0 < 32 ? X::template cols<32>(m, 0, s0) : X::template cols<64>(m + kUpper, 0, s0);
  }
};

constexpr int kBufWord3 = 0x00020000;  // raw buffer access, gfx9 family

// `bytes` bytes from p on: loads behind them give zeros, stores there nothing.
// Both are the same in all lanes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  const uint64_t u = (uint64_t)uniform_u32((uint32_t)(a >> 32)) << 32 | uniform_u32((uint32_t)a);
  return __builtin_amdgcn_make_buffer_rsrc((void*)u, 0, uniform_u32(bytes), kBufWord3);
}

__device__ __forceinline__ float buffer_float(__amdgpu_buffer_rsrc_t b, int lane_byte, int byte) {
  const uint32_t u = __builtin_amdgcn_raw_buffer_load_b32(b, lane_byte, byte, 0);
  return __uint_as_float(u);
}

// One [kChunk, D] block of a [T, D] array: 16-byte pieces through registers
// into an LDS matrix, zeros behind the last step.
template <class T, int D, int THREADS>
struct Block {
  static constexpr int kC = Tile<T>::kChunk;
  static constexpr int kSize = kC * Tile<T>::template kLd<D>;
  static constexpr int kRowPieces = D * (int)sizeof(T) / 16;
  static constexpr int kPieces = kC * kRowPieces;
  static constexpr int kN = (kPieces + THREADS - 1) / THREADS;
  u32x4 r[kN];

  __device__ __forceinline__ void load(const T* base, int valid_rows) {
    const __amdgpu_buffer_rsrc_t b = buffer(base, (uint32_t)(valid_rows * D * (int)sizeof(T)));
#pragma unroll
    for (int i = 0; i < kN; ++i)
      r[i] = __builtin_amdgcn_raw_buffer_load_b128(b, (threadIdx.x + i * THREADS) * 16, 0, 0);
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int p = threadIdx.x + i * THREADS;
      if ((i + 1) * THREADS <= kPieces || p < kPieces)
        *reinterpret_cast<u32x4*>(lds + Tile<T>::template at<D>(p / kRowPieces,
                                                                (p % kRowPieces) *
                                                                    (16 / (int)sizeof(T)))) = r[i];
    }
  }
};

// Waits for loads that are on their way into x.  (At a loop's entry: the
// compiler waits for registers loaded before a loop inside it, and so for the
// loads that the loop has just sent out.)
template <int N>
__device__ __forceinline__ void arrive(f32x4 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
}

// Orders of the instructions of a stretch of code between two calls of
// schedule_end(): the next n LDS reads, matrix instructions, writes to memory.
template <int N>
__device__ __forceinline__ void schedule_reads() {
  __builtin_amdgcn_sched_group_barrier(0x100, N, 0);
}
template <int N>
__device__ __forceinline__ void schedule_products() {
  __builtin_amdgcn_sched_group_barrier(0x008, N, 0);
}
template <int N>
__device__ __forceinline__ void schedule_writes() {
  __builtin_amdgcn_sched_group_barrier(0x040, N, 0);
}
__device__ __forceinline__ void schedule_end() { __builtin_amdgcn_sched_barrier(0); }

// Decays of one chunk.  The sums of logarithms are formed in 64 bits and kept
// as two floats, so that the decay between two steps has fp32's precision
// whatever other steps of the chunk forget.
template <int C>
struct alignas(16) Decays {
  float hi[C], lo[C];  // log2 of the decay from the chunk's start through step t
  float into[C];       // that decay
  float onto[C];       // decay behind step t to the chunk's end
  float whole;         // of the whole chunk
};

// 2^x, 0 below 2^-126
__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

// log2 of one step's decay.  At or below exp(-128) the step forgets the state: -1024,
// so that its sum with steps on both sides, whose own stretches stay below 2^128, is
// far below 2^-149 and the decay across it exactly 0.  (The sums of a chunk's
// 64 such steps keep 2^-33 beside 2^16.)
__device__ __forceinline__ double log2_decay(float g) {
  return g <= -128.0f ? -1024.0 : (double)g * 1.4426950408889634;
}

// x of the lane that the control kDpp names (in a row of 16), 0 where there is none
template <int kDpp>
__device__ __forceinline__ float row_move(float x) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), kDpp, 0xF, 0xF, true));
}
template <int kDpp>
__device__ __forceinline__ double row_move(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, kDpp, 0xF, 0xF, true);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), kDpp, 0xF, 0xF, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// of lane l - N, of lane l + N
template <int N, class F>
__device__ __forceinline__ F row_shr(F x) {
  return row_move<0x110 + N>(x);
}
template <int N, class F>
__device__ __forceinline__ F row_shl(F x) {
  return row_move<0x100 + N>(x);
}

// Sums over a row of 16 lanes, of the lanes up to this one and from this one on.
template <class F>
__device__ __forceinline__ F row_sums_down(F x) {
  x += row_shr<1>(x);
  x += row_shr<2>(x);
  x += row_shr<4>(x);
  x += row_shr<8>(x);
  return x;
}
template <class F>
__device__ __forceinline__ F row_sums_up(F x) {
  x += row_shl<1>(x);
  x += row_shl<2>(x);
  x += row_shl<4>(x);
  x += row_shl<8>(x);
  return x;
}

__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Sum of the lanes up to this one (of C lanes, by the whole wavefront); sum: of
// all C.  Lanes at or past C hold 0.
template <int C>
__device__ __forceinline__ double prefix_sum(double x, double& sum) {
  x = row_sums_down(x);
  double below = 0.0;
  sum = lane_value(x, 15);
#pragma unroll
  for (int r = 1; r < C / 16; ++r) {
    if (lane_id() >> 4 == r) below = sum;
    sum += lane_value(x, r * 16 + 15);
  }
  return x + below;
}

// By one whole wavefront, step `lane`'s x (0 behind the last step and in lanes
// at or past C): fills d and returns the chunk's sum.  onto and into reach
// further by the logarithms `behind` and `before` the chunk.
template <int C>
__device__ __forceinline__ double scan_decays(double x, Decays<C>& d, double before = 0.0,
                                              double behind = 0.0) {
  const int l = lane_id();
  double sum;
  x = prefix_sum<C>(x, sum);
  if (l < C) {
    const float hi = (float)x;
    d.hi[l] = hi;
    d.lo[l] = (float)(x - (double)hi);
    d.into[l] = pow2((float)(before + x));
    d.onto[l] = pow2((float)(behind + (sum - x)));
    if (l == 0) d.whole = pow2((float)sum);
  }
  return sum;
}

// decays behind steps s .. s + 3 through step t, 0 for steps behind t
template <int C>
__device__ __forceinline__ f32x4 decay_between(const Decays<C>& d, int t, int s) {
  const f32x4 hi = *reinterpret_cast<const f32x4*>(d.hi + s);
  const f32x4 lo = *reinterpret_cast<const f32x4*>(d.lo + s);
  const float thi = d.hi[t], tlo = d.lo[t];
  f32x4 x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float e = pow2((thi - hi[j]) + (tlo - lo[j]));
    x[j] = s + j <= t ? e : 0.0f;
  }
  return x;
}

// p * decay where there is one: what later steps hold (their decay is 0) does
// not enter
__device__ __forceinline__ f32x4 decayed(f32x4 p, f32x4 decay, int t, int s) {
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = s + j <= t ? p[j] * decay[j] : 0.0f;
  return p;
}

// A contiguous range of memories per XCD (workgroups go to the 8 XCDs in turn),
// so that heads that share keys share an L2.
__device__ __forceinline__ uint32_t xcd_contiguous(uint32_t block, uint32_t n) {
  return n % 8 == 0 ? (block & 7) * (n / 8) + (block >> 3) : block;
}

}  // namespace lin
}  // namespace sdm
