// Root-mean-square norms before and after a block, with the gate and the
// residual that go with them, and their gradients.  Per row y of d values:
//   r = 1 / sqrt(mean(y^2) + eps),  out = x + scale * silu(z) * w * y r
// and, if asked for, the next block's norm of the same row before out is
// rounded.  With n = y r, a = silu(z), s = sigmoid(z), D = scale * dout:
//   dz = D n w s (1 + z (1 - s)),   dw = sum over rows of D a n
//   dy = r (D a w - n mean(D a w n)) + skip
// Rows of y come as the block's outputs do: [rows, d], or [B, H, T, d] whose
// outputs are wanted as [B, T, H d].
//
// Bound by memory: every value is read once into registers (8 at a time per
// lane), sums are fp32.  Rows of up to 512 values take a power of two of lanes,
// 256-thread workgroups several rows; longer rows take a workgroup each.  Measured:
//   8192 rows of 8192 bf16 with gate, residual and next norm (671 MB) 130-138 us,
//     4.9-5.2 TB/s (a copy of that mix, three arrays read and one written, 5.6);
//   262144 rows of 128, fp32 to gated bf16 by heads (268 MB) 50 us, 5.4 TB/s;
//   their reverse pass, 131072 rows of bf16 (168 MB) and the sum of dw, 34-39 + 4 us;
//     in fp32 66-71 + 5;
//   4099 rows of 5128, fp32 from bf16 gradients (294 MB), 66 + 6 us, 4.4 TB/s;
//   reverse, whole rows of 16384, bf16, 4096 of them (537 MB) 122 + 7 us, 4.4 TB/s;
//     fp32, 2048 of them (537 MB) 108-114 + 7, 4.7-5.0;
//   without a gate, 32768 rows of 4096 bf16 or 8192 of 8192 fp32 (537 MB) 101 us, 5.3;
//   one row of 8192 3 us.
#include "dense.h"
#include "device_common.h"

namespace sdm {
namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kNarrow = 256;      // threads of a workgroup of short rows
constexpr int kNarrowMax = 512;   // values of a short row
constexpr int kWideMax = 1024;    // threads of a long row
constexpr int kFewRows = 512;

// Eight values of a row, read or written once: past the caches (8192 rows of
// 8192 with gate, residual and next norm 135 us with ordinary accesses, 126).
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 r;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    r = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const uint16_t*)p + at));
  }
  __device__ __forceinline__ f32x8 values() const {
    return __builtin_convertvector(__builtin_bit_cast(bf16x8, r), f32x8);
  }
};
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const f32x4* f = reinterpret_cast<const f32x4*>((const float*)p + at);
    a = __builtin_nontemporal_load(f);
    b = __builtin_nontemporal_load(f + 1);
  }
  __device__ __forceinline__ f32x8 values() const {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

template <class T>
__device__ __forceinline__ f32x8 load8(const void* p, int64_t at) {
  Raw8<T> r;
  r.load(p, at);
  return r.values();
}

template <class T>
__device__ __forceinline__ void store8(void* p, int64_t at, f32x8 v) {
  if constexpr (sizeof(T) == 2) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, __builtin_convertvector(v, bf16x8)),
                                reinterpret_cast<u32x4*>((uint16_t*)p + at));
  } else {
    f32x4* f = reinterpret_cast<f32x4*>((float*)p + at);
    __builtin_nontemporal_store(__builtin_shufflevector(v, v, 0, 1, 2, 3), f);
    __builtin_nontemporal_store(__builtin_shufflevector(v, v, 4, 5, 6, 7), f + 1);
  }
}

// Eight values that are read again soon.
__device__ __forceinline__ void put8(float* p, int at, f32x8 v) {
  f32x4* f = reinterpret_cast<f32x4*>(p + at);
  f[0] = __builtin_shufflevector(v, v, 0, 1, 2, 3);
  f[1] = __builtin_shufflevector(v, v, 4, 5, 6, 7);
}

// Eight weights, which every row reads.
__device__ __forceinline__ f32x8 weights8(const float* p, int at) {
  const f32x4* f = reinterpret_cast<const f32x4*>(p + at);
  return __builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ float sum8(f32x8 v) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// 1 / (1 + exp(-z)), from the hardware's 2^x and 1/x (each within an ulp): a
// row's gates cost more than its other arithmetic.  The exponent t = -z log2 e,
// rounded, is off by up to 2^-24 of itself, which the power would multiply by z:
// what t lacks, r, is put back as the factor 2^r = 1 + r ln 2.  Beyond the bounds
// of z the result is 0 or 1 anyway, and r stays small.
__device__ __forceinline__ float sigmoid(float z) {
  constexpr float kL = -1.44269504088896f;       // -log2 e, and the rest of it
  constexpr float kRest = (float)(-1.4426950408889634 - (double)kL);
  z = __builtin_amdgcn_fmed3f(z, -104.0f, 88.0f);
  const float t = z * kL;
  const float r = __builtin_fmaf(z, kRest, __builtin_fmaf(z, kL, -t));
  const float e = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(r, 0.693147181f, 1.0f);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// Sums of N values over a row's lanes: `lanes` of them (a power of two up to 64)
// or, WIDE, the whole workgroup.  Every lane gets the same bits.
template <bool WIDE, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int lanes, float (*lds)[kWideMax / kWave]) {
  if (!WIDE) {
    for (int o = 1; o < lanes; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = wave_sum_f32(v[i]);
    if (lane_id() == 0) lds[i][threadIdx.x / kWave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lds[i][0];
  for (int w = 1; w < (int)(blockDim.x / kWave); ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += lds[i][w];
  __syncthreads();  // lds is free again
}

// Sum over a long row of what each thread has for its V vectors, by pieces of 64
// vectors in their order: the same bits for one vector a thread and for two.
template <int V>
__device__ __forceinline__ float long_row_sum(const float (&v)[V], float* lds) {
  const int waves = (int)(blockDim.x / kWave);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float s = wave_sum_f32(v[i]);
    if (lane_id() == 0) lds[i * waves + threadIdx.x / kWave] = s;
  }
  __syncthreads();
  float sum = lds[0];
  for (int w = 1; w < V * waves; ++w) sum += lds[w];
  __syncthreads();  // lds is free again
  return sum;
}

// Row r of the outputs (b, t, h), as a row of y.
__device__ __forceinline__ int64_t y_row(const NormArgs& A, uint32_t r) {
  if (A.H == 1) return r;
  const uint32_t H = A.H, T = (uint32_t)A.T;
  const uint32_t bt = A.by_h.of(r), h = r - bt * H, b = A.by_t.of(bt), t = bt - b * T;
  return ((int64_t)b * H + h) * T + t;
}

template <class Ty, class To, int V, bool WIDE>
__global__ __launch_bounds__(WIDE ? kWideMax : kNarrow) void norm_kernel(NormArgs A, int lanes) {
// A row's bits do not depend on the variant that takes it: the kernel's products
// and sums are rounded as they stand (the compiler might fuse them differently).
#pragma clang fp contract(off)
  __shared__ float lds[WIDE ? V * kWideMax / kWave : 1];
  const int nvec = A.d / 8;
  const int group = WIDE ? 0 : threadIdx.x / lanes, me = WIDE ? threadIdx.x : threadIdx.x % lanes;
  const int per_block = WIDE ? 1 : kNarrow / lanes, L = WIDE ? (int)blockDim.x : lanes;
  const auto row_sum = [&](float (&v)[V]) {
    if constexpr (WIDE) return long_row_sum(v, lds);
    for (int o = 1; o < lanes; o <<= 1) v[0] += __shfl_xor(v[0], o);
    return v[0];
  };
  // every lane of a wavefront runs the same passes (the sums exchange lanes)
  for (int64_t r0 = (int64_t)blockIdx.x * per_block; r0 < A.rows;
       r0 += (int64_t)gridDim.x * per_block) {
    const int64_t r = r0 + group;
    const bool here = r < A.rows;
    const int64_t yr = here ? y_row(A, (uint32_t)r) * A.d : 0, at = r * A.d;
    f32x8 y[V];
    float ss[V];  // squares, by vectors
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = me + i * L;
      y[i] = here && j < nvec ? load8<Ty>(A.y, yr + j * 8) : f32x8{0, 0, 0, 0, 0, 0, 0, 0};
    }
    f32x8 z[V], x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = me + i * L;
      if (here && j < nvec) {
        if (A.z) z[i] = load8<To>(A.z, at + j * 8);
        if (A.x) x[i] = load8<To>(A.x, at + j * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) ss[i] = sum8(y[i] * y[i]);
    const float rs = A.scale / sqrtf(row_sum(ss) / (float)A.d + A.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = me + i * L;
      ss[i] = 0.0f;
      if (!here || j >= nvec) continue;
      y[i] = y[i] * rs * weights8(A.w, j * 8);
      if (A.z) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] *= z[i][e] * sigmoid(z[i][e]);
      }
      if (A.x) y[i] += x[i];
      store8<To>(A.out, at + j * 8, y[i]);
      ss[i] = sum8(y[i] * y[i]);
    }
    if (A.next_w) {
      const float rn = 1.0f / sqrtf(row_sum(ss) / (float)A.d + A.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = me + i * L;
        if (here && j < nvec) store8<To>(A.next, at + j * 8, y[i] * rn * weights8(A.next_w, j * 8));
      }
    }
  }
}

// Each workgroup takes rows blockIdx, blockIdx + blocks, ... and leaves its
// sum of dw in part[blockIdx].  A lane's vector of a bf16 row (eight registers
// with its gate and gradients) is loaded as it stands, all arrays in one go (131072
// gated rows of 128 39 us, 42 as separate values), and for long rows before the
// sums of the row in front of it (20000 of 2048 64 us, 71).  fp32 rows and two
// vectors a thread have the registers for that only at half the workgroups (4099
// rows of 5128 76-84 us for 72; 32768 fp32 rows of 256 109 for 103).
template <class Ty, class To, int V, bool WIDE>
__global__ __launch_bounds__(WIDE ? kWideMax / 2 : kNarrow) void norm_backward_kernel(NormArgs A,
                                                                                   int lanes) {
  constexpr bool kRaw = V == 1 && sizeof(Ty) + sizeof(To) == 4, kAhead = kRaw && WIDE;
  __shared__ float lds[2][kWideMax / kWave];
  __shared__ __align__(16) float sum[WIDE ? 8 : kNarrow * 8];
  const int nvec = A.d / 8;
  const int group = WIDE ? 0 : threadIdx.x / lanes, me = WIDE ? threadIdx.x : threadIdx.x % lanes;
  const int per_block = WIDE ? 1 : kNarrow / lanes, L = WIDE ? (int)blockDim.x : lanes;
  f32x8 w[V], dw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = me + i * L;
    dw[i] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
    w[i] = j < nvec ? weights8(A.w, j * 8) : dw[i];
  }
  Raw8<Ty> next_y, next_skip;  // kRaw
  Raw8<To> next_dout, next_z;
  const auto fetch = [&](int64_t r) {
    if (r >= A.rows || me >= nvec) return;
    const int64_t yr = y_row(A, (uint32_t)r) * A.d, at = r * A.d;
    next_y.load(A.y, yr + me * 8);
    next_dout.load(A.dout, at + me * 8);
    if (A.z) next_z.load(A.z, at + me * 8);
    if (A.skip) next_skip.load(A.skip, yr + me * 8);
  };
  if (kAhead) fetch(blockIdx.x);
  for (int64_t r0 = (int64_t)blockIdx.x * per_block; r0 < A.rows;
       r0 += (int64_t)gridDim.x * per_block) {
    const int64_t r = r0 + group;
    const bool here = r < A.rows;
    const int64_t yr = here ? y_row(A, (uint32_t)r) * A.d : 0, at = r * A.d;
    f32x8 y[V], D[V], z[V];
    f32x8 gate;  // the sigmoids, where registers allow (V = 1)
    if (kRaw && !kAhead) fetch(r);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = me + i * L;
      const bool in = here && j < nvec;
      const f32x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
      if (kRaw) {
        y[i] = in ? next_y.values() : zero;
        D[i] = in ? next_dout.values() * A.scale : zero;
        z[i] = in && A.z ? next_z.values() : zero;
      } else {
        y[i] = in ? load8<Ty>(A.y, yr + j * 8) : zero;
        D[i] = in ? load8<To>(A.dout, at + j * 8) * A.scale : zero;
        z[i] = in && A.z ? load8<To>(A.z, at + j * 8) : zero;
      }
    }
    const Raw8<Ty> skip = next_skip;
    if (kAhead) fetch(r0 + gridDim.x);
    float sums[2] = {0.0f, 0.0f};  // y^2, D a w y
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f32x8 a = D[i] * w[i];
      if (A.z) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = sigmoid(z[i][e]);
          if (V == 1) gate[e] = s;
          a[e] *= z[i][e] * s;
        }
      }
      sums[0] += sum8(y[i] * y[i]);
      sums[1] += sum8(a * y[i]);
    }
    row_sums<WIDE>(sums, lanes, lds);
    const float rs = 1.0f / sqrtf(sums[0] / (float)A.d + A.eps);
    const float mean = sums[1] * rs / (float)A.d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = me + i * L;
      if (!here || j >= nvec) continue;
      const f32x8 n = y[i] * rs;
      f32x8 a = D[i];
      if (A.z) {
        f32x8 dz;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = V == 1 ? gate[e] : sigmoid(z[i][e]);
          dz[e] = D[i][e] * n[e] * w[i][e] * (s * (1.0f + z[i][e] * (1.0f - s)));
          a[e] *= z[i][e] * s;
        }
        store8<To>(A.dz, at + j * 8, dz);
      }
      dw[i] += a * n;
      f32x8 dy = (a * w[i] - n * mean) * rs;
      if (A.skip) dy += kRaw ? skip.values() : load8<Ty>(A.skip, yr + j * 8);
      store8<Ty>(A.dy, yr + j * 8, dy);
    }
  }
  float* part = A.part + (int64_t)blockIdx.x * A.d;
  if (WIDE) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (me + i * L < nvec) put8(part, (me + i * L) * 8, dw[i]);
    return;
  }
  put8(sum, threadIdx.x * 8, dw[0]);
  __syncthreads();
  if (group == 0 && me < nvec) {
    for (int k = 1; k < per_block; ++k) dw[0] += weights8(sum, (k * lanes + me) * 8);
    put8(part, me * 8, dw[0]);
  }
}

// dw = sum of the workgroups' parts, in a fixed order: 4 * LANES columns a
// workgroup, 256 / LANES parts at a time, four of them in flight.
template <int LANES>
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* part, float* dw, int d,
                                                      int blocks) {
  constexpr int kRows = 256 / LANES;
  __shared__ f32x4 lds[kRows][LANES];
  const int cl = threadIdx.x % LANES, rl = threadIdx.x / LANES;
  const int c = (blockIdx.x * LANES + cl) * 4;
  const f32x4 zero = {0, 0, 0, 0};
  f32x4 s = zero;
  if (c < d)
    for (int b = rl; b < blocks; b += 4 * kRows) {
      f32x4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = b + i * kRows;
        v[i] = *reinterpret_cast<const f32x4*>(part + (int64_t)(r < blocks ? r : b) * d + c);
        if (r >= blocks) v[i] = zero;
      }
      s += (v[0] + v[1]) + (v[2] + v[3]);
    }
  lds[rl][cl] = s;
  __syncthreads();
  for (int n = kRows / 2; n > 0; n /= 2) {
    if (rl < n) lds[rl][cl] += lds[rl + n][cl];
    __syncthreads();
  }
  if (rl == 0 && c < d) *reinterpret_cast<f32x4*>(dw + c) = lds[0][cl];
}

int row_lanes(int d) {  // of a short row
  int lanes = 1;
  while (lanes * 8 < d) lanes *= 2;
  return lanes;
}

// n / d for n below 2^31: 2^(31 + l) / d rounded up, l = ceil(log2 d), is below
// 2^32 and exceeds the quotient by less than 2^l, so n times it is off by less
// than 1 / d.
NormDivisor divisor(uint32_t d) {
  NormDivisor v;
  v.shift = 31;
  while (((uint64_t)1 << (v.shift - 31)) < d) ++v.shift;
  v.mul = (uint32_t)((((uint64_t)1 << v.shift) + d - 1) / d);
  return v;
}

void set_divisors(NormArgs& a) {
  if (a.H == 1) return;
  a.by_h = divisor((uint32_t)a.H);
  a.by_t = divisor((uint32_t)(a.T < 1 ? 1 : a.T));
}

int wide_threads(int d, int V) { return (d / 8 + V * kWave - 1) / (V * kWave) * kWave; }

template <class Ty, class To>
hipError_t norm_types(const NormArgs& a, hipStream_t s) {
  constexpr int64_t kMaxBlocks = (int64_t)1 << 20;
  if (a.d <= kNarrowMax) {
    const int lanes = row_lanes(a.d);
    const int64_t want = (a.rows + kNarrow / lanes - 1) / (kNarrow / lanes);
    const int64_t blocks = want < kMaxBlocks ? want : kMaxBlocks;
    hipLaunchKernelGGL((norm_kernel<Ty, To, 1, false>), dim3((unsigned)blocks), dim3(kNarrow), 0, s,
                       a, lanes);
    return hipGetLastError();
  }
  const dim3 blocks((unsigned)(a.rows < kMaxBlocks ? a.rows : kMaxBlocks));
  // few rows: a row's latency counts, so as many threads as it has vectors (256 rows
  // of 4096 bf16 6.1 us, 8.0 with two a thread; 512 of 8192 11.5, 12.0); otherwise
  // two vectors a thread (8192 rows of 8192, replayed from a graph, 134 us, one 137;
  // 16384 of 4096 55.8, one 58.5; fp32 rows the other way, 133 and 129)
  if (a.rows <= kFewRows && a.d <= 8 * kWideMax)
    hipLaunchKernelGGL((norm_kernel<Ty, To, 1, true>), blocks, dim3(wide_threads(a.d, 1)), 0, s, a, 0);
  else
    hipLaunchKernelGGL((norm_kernel<Ty, To, 2, true>), blocks, dim3(wide_threads(a.d, 2)), 0, s, a, 0);
  return hipGetLastError();
}

template <class Ty, class To>
hipError_t norm_backward_types(const NormArgs& a, hipStream_t s) {
  const int64_t n = norm_backward_blocks(a.rows, a.d);
  const dim3 blocks((unsigned)n);
  if (n == 0)
    ;  // no rows: dw is 0
  else if (a.d <= kNarrowMax)
    hipLaunchKernelGGL((norm_backward_kernel<Ty, To, 1, false>), blocks, dim3(kNarrow), 0, s, a,
                       row_lanes(a.d));
  else if (a.d <= 8 * 512)
    hipLaunchKernelGGL((norm_backward_kernel<Ty, To, 1, true>), blocks, dim3(wide_threads(a.d, 1)),
                       0, s, a, 0);
  else if (a.d <= 8 * 1024)
    hipLaunchKernelGGL((norm_backward_kernel<Ty, To, 2, true>), blocks, dim3(wide_threads(a.d, 2)),
                       0, s, a, 0);
  else
    hipLaunchKernelGGL((norm_backward_kernel<Ty, To, 4, true>), blocks, dim3(wide_threads(a.d, 4)),
                       0, s, a, 0);
  hipError_t rc = hipGetLastError();
  if (rc != hipSuccess) return rc;
  // few columns: as many workgroups as there are 16-byte pieces (128 columns of
  // 1024 parts 7 us with 16 columns a workgroup)
  if (a.d <= kNarrowMax)
    hipLaunchKernelGGL(norm_dw_kernel<1>, dim3((unsigned)(a.d / 4)), dim3(256), 0, s, a.part, a.dw,
                       a.d, (int)n);
  else
    hipLaunchKernelGGL(norm_dw_kernel<4>, dim3((unsigned)((a.d + 15) / 16)), dim3(256), 0, s,
                       a.part, a.dw, a.d, (int)n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(NormArgs a, int y_dtype, int out_dtype, hipStream_t s) {
  set_divisors(a);
  if (y_dtype == 1)
    return out_dtype == 1 ? norm_types<uint16_t, uint16_t>(a, s) : norm_types<uint16_t, float>(a, s);
  return out_dtype == 1 ? norm_types<float, uint16_t>(a, s) : norm_types<float, float>(a, s);
}

// Workgroups of the reverse pass, each of which leaves d partial sums: as many
// as are resident together (16 wavefronts a compute unit, 8 with four vectors a
// thread).  4099 rows of 5128: 512 of them 66 us, 682 (a second round) 82.
int64_t norm_backward_blocks(int64_t rows, int d) {
  const bool narrow = d <= kNarrowMax;
  const int V = narrow || d <= 8 * 512 ? 1 : d <= 8 * 1024 ? 2 : 4;
  const int waves = (narrow ? kNarrow : wide_threads(d, V)) / kWave;
  const int per_block = narrow ? kNarrow / row_lanes(d) : 1;
  const int64_t want = (rows + per_block - 1) / per_block, most = 256 * ((V == 4 ? 8 : 16) / waves);
  return want < most ? want : most;
}

hipError_t launch_norm_backward(NormArgs a, int y_dtype, int out_dtype, hipStream_t s) {
  set_divisors(a);
  if (y_dtype == 1)
    return out_dtype == 1 ? norm_backward_types<uint16_t, uint16_t>(a, s)
                          : norm_backward_types<uint16_t, float>(a, s);
  return out_dtype == 1 ? norm_backward_types<float, uint16_t>(a, s)
                        : norm_backward_types<float, float>(a, s);
}

}  // namespace sdm
