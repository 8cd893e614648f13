// Reverse pass from the 8-bit tape (mx.h, 8-bit form): the gradients of
// backward.hip (page "Riepilogo Tecnico: Sparse Delta Memory (SDM)", section
// "Meccanismo Core", items 3 and 4), organised around what the small tape
// makes cheap.  Per step t, in reverse (backward.hip states the formulas):
//   dr_l = <do, M_t[g_l]>                    needs the tape alone;
//   G[g_l] += r_l do;  g = G[f_j];           the recurrence through G;
//   dv, dalpha, d(beta k_j) from g and the tape's pre-write rows;
//   G[f_j] = alpha (1 - beta k_j) g.
//
// Three kernels:
//   prepare  one wavefront per step, all steps at once: dr from the tape's
//            read rows, and the step's record for the scan -- the byte offsets
//            of its rows of G, the read weight that falls on each write row
//            (the row's own, when the step also reads it), k_j, and
//            whether any of its rows is also touched by the step after it in
//            time, i.e. just before it in the scan;
//   scan     one workgroup per (memory, column tile) walks the records.  Its
//            second wavefront streams them into LDS two chunks ahead, so the
//            first spends its instructions on G: it gathers a step's rows of G
//            and its pre-write rows while it computes the step before, updates,
//            reduces and stores.  The gathers go out before that step's
//            stores; a step whose record says that they touch the same rows
//            gathers again after them (never wrong, and rare while the table
//            is much larger than a step's rows);
//   finish   adds the tiles' partial sums in a fixed order.
// Scales are powers of two, so the whole numbers of a tape row enter a sum as
// they are and the block's scale multiplies the sum.
#include "internal.h"
#include "mx.h"
#include "ranges.h"

namespace sdm {
namespace {

constexpr int kBufWord3 = 0x00020000;  // raw buffer access, gfx9 family
constexpr uint32_t kOffNone = ranges::kOffNone;

constexpr int kChunk = 8;  // records per LDS chunk
constexpr int kRing = 3;

// A step's record.  Row entries are transposed for the tile width in use:
// entry lr * NI + k is row slot k * RPI + lr.  Offsets are multiples of 64
// (whole rows); bit 0 marks a row whose gradient is still zero (sparse mode:
// its last touch in time), which is stored but not gathered.
struct Record {
  uint32_t wofs[64];
  uint32_t rofs[64];
  float mw[64];
  float rw[64];
  float wk[64];
  float alpha, beta;
  uint32_t again;  // rows shared with the record before this one
  uint32_t pad;
};
static_assert(sizeof(Record) % 16 == 0, "records move in 16-byte pieces");

// Records are numbered in reverse time, u = T - 1 - t, and end with at least
// one that has no rows.
__host__ __device__ inline int64_t padded_steps(int64_t T) { return (T + kChunk) / kChunk * kChunk; }

struct Bwd8Args {
  int n_mem;
  int64_t N;
  int d_v;
  int64_t T;
  int W, R;
  const int32_t* widx;
  const float* wk;
  const int32_t* ridx;
  const float* rw;
  const float* v;
  const float* alpha;
  const float* beta;
  const float* dout;
  const int8_t* tape;
  const uint8_t* tape_scale;
  float* G;
  float *dv, *dwk, *drw, *dalpha, *dbeta;
  const uint64_t* first;
  Record* rec;  // [n_mem, padded_steps(T)]
  float* sums;  // [n_mem, T, ntiles, W + 1]: per tile d(beta k), then dalpha
  int ntiles, cols;
};

// ---------------------------------------------------------------- prepare

__global__ __launch_bounds__(256) void prepare_kernel(Bwd8Args A) {
  const int64_t Tp = padded_steps(A.T);
  const int64_t unit = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (unit >= (int64_t)A.n_mem * Tp) return;  // whole wavefront leaves together
  const int64_t mem = unit / Tp, u = unit - mem * Tp, t = A.T - 1 - u;
  const int lane = lane_id(), W = A.W, R = A.R;
  Record& out = A.rec[unit];
  const int lpr = A.cols / 4, rpi = kWave / lpr, ni = 64 / rpi;
  const int at = (lane % rpi) * ni + lane / rpi;  // this lane's slot in the record
  if (t < 0) {
    out.wofs[at] = kOffNone;
    out.rofs[at] = kOffNone;
    if (lane == 0) out.again = 0;
    return;
  }
  const int64_t step = mem * A.T + t;
  const uint32_t N = (uint32_t)A.N, row_bytes = (uint32_t)A.d_v * 4u;
  // rows outside the table: all ones, which no row number equals
  auto row = [&](const int32_t* idx, int K, int64_t s) __attribute__((always_inline)) {
    const uint32_t r = lane < K ? (uint32_t)idx[s * K + lane] : ~0u;
    return r < N ? r : ~0u;
  };
  const uint32_t w = row(A.widx, W, step), r = row(A.ridx, R, step);
  const float wk = lane < W ? A.wk[step * W + lane] : 0.0f;
  const float rw = lane < R ? A.rw[step * R + lane] : 0.0f;
  const uint64_t fw = A.first ? A.first[step * 2] : 0ull, fr = A.first ? A.first[step * 2 + 1] : 0ull;

  // the read weight that falls on a write row
  float mw = 0.0f;
  for (int l = 0; l < R; ++l) {
    const uint32_t s = (uint32_t)__builtin_amdgcn_readlane((int)r, l);
    const float x = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(rw), l));
    if (w == s) mw = x;
  }
  if (w == ~0u) mw = 0.0f;
  // rows shared with step t + 1
  bool again = false;
  if (u > 0) {
    const uint32_t w1 = row(A.widx, W, step + 1), r1 = row(A.ridx, R, step + 1);
    for (int l = 0; l < W; ++l) {
      const uint32_t s = (uint32_t)__builtin_amdgcn_readlane((int)w1, l);
      again |= s != ~0u && (w == s || r == s);
    }
    for (int l = 0; l < R; ++l) {
      const uint32_t s = (uint32_t)__builtin_amdgcn_readlane((int)r1, l);
      again |= s != ~0u && (w == s || r == s);
    }
  }
  const bool shared = __ballot(again) != 0ull;
  out.wofs[at] = w == ~0u ? kOffNone : w * row_bytes | (uint32_t)((fw >> lane) & 1ull);
  out.rofs[at] = r == ~0u ? kOffNone : r * row_bytes | (uint32_t)((fr >> lane) & 1ull);
  out.mw[at] = mw;
  out.rw[at] = rw;
  out.wk[at] = wk;
  if (lane == 0) {
    out.alpha = A.alpha[step];
    out.beta = A.beta[step];
    out.again = shared ? 1u : 0u;
  }

  // dr: lane l's read row, block by block, against the step's output gradient
  if (lane < R) {
    const int nb = A.d_v / 16;
    const int64_t S = A.T * (W + R);
    float dr = 0.0f;
    if (r != ~0u) {
      for (int b = 0; b < nb; ++b) {
        const int64_t rec = (mem * nb + b) * S + t * (W + R) + W + lane;
        const u32x4 q = *reinterpret_cast<const u32x4*>(A.tape + rec * 16);
        const uint32_t c[4] = {q.x, q.y, q.z, q.w};
        const float* d = A.dout + step * A.d_v + b * 16;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[4];
          int8_unpack4(c[i], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) s = fmaf(d[4 * i + e], x[e], s);
        }
        dr = fmaf(s, __uint_as_float((uint32_t)A.tape_scale[rec] << 23), dr);
      }
    }
    A.drw[step * R + lane] = dr;
  }
}

// ---------------------------------------------------------------- scan

template <int COLS>
struct Lds8 {
  Record rec[kRing][kChunk];
  float vd[kRing][2][kChunk][COLS];  // the tile's columns of v and dout
};

__device__ __forceinline__ void chunk_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ f32x4 as_f4(const u32x4& q) {
  return f32x4{__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z),
               __uint_as_float(q.w)};
}
__device__ __forceinline__ u32x4 as_u4(const f32x4& f) {
  return u32x4{__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z),
               __float_as_uint(f.w)};
}

// Of two values per lane, the sum over the pair of lanes 1 << BIT apart of the
// one this lane's bit selects.
template <int BIT>
__device__ __forceinline__ float fold(float a, float b) {
  const bool up = lane_id() & (1 << BIT);
  const float keep = up ? b : a, send = up ? a : b;
  return keep + __uint_as_float(lane_xor(__float_as_uint(send), 1 << BIT));
}

template <int COLS>
struct Scan8 {
  static constexpr int LPR = COLS / 4, RPI = kWave / LPR, NI = 64 / RPI, NG = NI / 4;

  // A step in flight: its offsets, its rows of G and its pre-write records.
  struct Step {
    uint32_t wo[NI], ro[NI];
    u32x4 Gw[NI], Gr[NI];
    u32x4 codes[NG];
    uint32_t scale[NG];
  };

  const Bwd8Args& A;
  Lds8<COLS>& sh;
  __amdgpu_buffer_rsrc_t gres, tres, sres;
  uint32_t lane_off, rec0, step_rows;
  int lr, lc;
  int64_t T;

  __device__ __forceinline__ const Record& record(int64_t u) const {
    return sh.rec[(u / kChunk) % kRing][u % kChunk];
  }

  __device__ __forceinline__ void gather(Step& s) const {
#pragma unroll
    for (int k = 0; k < NI; ++k)
      s.Gr[k] = __builtin_amdgcn_raw_buffer_load_b128(
          gres, (s.ro[k] & 1u) ? kOffNone : s.ro[k] + lane_off, 0, 0);
#pragma unroll
    for (int k = 0; k < NI; ++k)
      s.Gw[k] = __builtin_amdgcn_raw_buffer_load_b128(
          gres, (s.wo[k] & 1u) ? kOffNone : s.wo[k] + lane_off, 0, 0);
  }

  __device__ __forceinline__ void issue(Step& s, int64_t u) const {
    const Record& r = record(u);
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      s.wo[k] = r.wofs[lr * NI + k];
      s.ro[k] = r.rofs[lr * NI + k];
    }
    gather(s);
    // lane q of a quad: the record of slot (4 g + q) * RPI + lr in the quad's block
    const int q = lane_id() & 3;
    const uint32_t row0 = rec0 + (uint32_t)(T - 1 - u) * step_rows;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const bool none = r.wofs[lr * NI + 4 * g + q] >= kOffNone;
      const uint32_t rec = row0 + (uint32_t)(4 * g * RPI);
      s.codes[g] = __builtin_amdgcn_raw_buffer_load_b128(tres, none ? kOffNone : rec * 16u, 0, 0);
      s.scale[g] = __builtin_amdgcn_raw_buffer_load_b8(sres, none ? kOffNone : rec, 0, 0);
    }
  }

  // Step u, with step u + 1's loads going out first.
  __device__ __forceinline__ void step(Step& s, Step& next, int64_t u, float* dv, float* sums) const {
    issue(next, u + 1);
    const Record& r = record(u);
    float rw[NI], mw[NI], wk[NI];
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      rw[k] = r.rw[lr * NI + k];
      mw[k] = r.mw[lr * NI + k];
      wk[k] = r.wk[lr * NI + k];
    }
    const float a = r.alpha, b = r.beta;
    const uint32_t again = record(u + 1).again;
    const int ring = (int)((u / kChunk) % kRing), at = (int)(u % kChunk);
    const f32x4 vv = *reinterpret_cast<const f32x4*>(&sh.vd[ring][0][at][lc * 4]);
    const f32x4 dd = *reinterpret_cast<const f32x4*>(&sh.vd[ring][1][at][lc * 4]);

    // ---- read rows: G += r do
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      f32x4 g = as_f4(s.Gr[k]);
      g.x = fmaf(rw[k], dd.x, g.x);
      g.y = fmaf(rw[k], dd.y, g.y);
      g.z = fmaf(rw[k], dd.z, g.z);
      g.w = fmaf(rw[k], dd.w, g.w);
      s.Gr[k] = as_u4(g);
    }
    // ---- write rows
    f32x4 dva = {0.f, 0.f, 0.f, 0.f};
    float da = 0.0f, dbk[NI];
#pragma unroll
    for (int g4 = 0; g4 < NG; ++g4) {
      // word i, after the exchange within the quad, is this lane's four
      // columns of slot (4 g4 + i) * RPI + lr; its scale is lane i's
      uint32_t w[4] = {s.codes[g4].x, s.codes[g4].y, s.codes[g4].z, s.codes[g4].w};
      quad_transpose(w);
      const float sc[4] = {__uint_as_float(dpp_mov<0x00>(s.scale[g4]) << 23),
                           __uint_as_float(dpp_mov<0x55>(s.scale[g4]) << 23),
                           __uint_as_float(dpp_mov<0xAA>(s.scale[g4]) << 23),
                           __uint_as_float(dpp_mov<0xFF>(s.scale[g4]) << 23)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 4 * g4 + i;
        float p[4];
        int8_unpack4(w[i], p);
        f32x4 g = as_f4(s.Gw[k]);
        g.x = fmaf(mw[k], dd.x, g.x);
        g.y = fmaf(mw[k], dd.y, g.y);
        g.z = fmaf(mw[k], dd.z, g.z);
        g.w = fmaf(mw[k], dd.w, g.w);
        const float bk = b * wk[k], keep = fmaf(-b, wk[k], 1.0f);
        dva.x = fmaf(bk, g.x, dva.x);
        dva.y = fmaf(bk, g.y, dva.y);
        dva.z = fmaf(bk, g.z, dva.z);
        dva.w = fmaf(bk, g.w, dva.w);
        const float gp = g.x * p[0] + g.y * p[1] + g.z * p[2] + g.w * p[3];
        da = fmaf(keep * sc[i], gp, da);
        const float ap = a * sc[i];
        dbk[k] = g.x * (vv.x - ap * p[0]) + g.y * (vv.y - ap * p[1]) +
                 g.z * (vv.z - ap * p[2]) + g.w * (vv.w - ap * p[3]);
        const float c = a * keep;
        s.Gw[k] = as_u4(f32x4{c * g.x, c * g.y, c * g.z, c * g.w});
      }
    }
    // ---- stores: read rows, then write rows (a row that is both ends with its
    // write-side value)
#pragma unroll
    for (int k = 0; k < NI; ++k)
      __builtin_amdgcn_raw_buffer_store_b128(s.Gr[k], gres, (s.ro[k] & ~1u) + lane_off, 0, 0);
#pragma unroll
    for (int k = 0; k < NI; ++k)
      __builtin_amdgcn_raw_buffer_store_b128(s.Gw[k], gres, (s.wo[k] & ~1u) + lane_off, 0, 0);

    // ---- the step's sums.  d(beta k): over the row's LPR lanes, folded so that
    // lane lc ends with the row of k = lc.
    float f[NI / 2];
#pragma unroll
    for (int i = 0; i < NI / 2; ++i) f[i] = fold<0>(dbk[2 * i], dbk[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < NI / 4; ++i) f[i] = fold<1>(f[2 * i], f[2 * i + 1]);
    if constexpr (NI == 8) f[0] = fold<2>(f[0], f[1]);
    const int j = lc * RPI + lr;
    if (j < A.W) sums[j] = f[0];
    // dv: over the lanes of the same columns; half wavefronts and rows of 16
    // are added two values at a time, so component (0, 2, 1, 3)[lane / 16] of
    // the lane's four columns stays
    {
      auto h0 = __builtin_amdgcn_permlane32_swap(__float_as_uint(dva.x), __float_as_uint(dva.y), false, false);
      auto h1 = __builtin_amdgcn_permlane32_swap(__float_as_uint(dva.z), __float_as_uint(dva.w), false, false);
      const float s0 = __uint_as_float(h0[0]) + __uint_as_float(h0[1]);
      const float s1 = __uint_as_float(h1[0]) + __uint_as_float(h1[1]);
      auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(s0), __float_as_uint(s1), false, false);
      float x = __uint_as_float(q[0]) + __uint_as_float(q[1]);
      x += __uint_as_float(dpp_row_ror8(__float_as_uint(x)));
      if constexpr (LPR == 4) x += __uint_as_float(dpp_row_ror4(__float_as_uint(x)));
      const int lane = lane_id(), row = lane >> 4;
      if ((lane & 15) < LPR) dv[(lane & 15) * 4 + ((row & 1) << 1 | row >> 1)] = x;
    }
    // dalpha: over the whole wavefront
    {
      float x = da;
      x += __uint_as_float(dpp_qp_xor1(__float_as_uint(x)));
      x += __uint_as_float(dpp_qp_xor2(__float_as_uint(x)));
      x += __uint_as_float(dpp_row_ror4(__float_as_uint(x)));
      x += __uint_as_float(dpp_row_ror8(__float_as_uint(x)));
      auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
      x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
      auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
      x = __uint_as_float(q[0]) + __uint_as_float(q[1]);
      if (lane_id() == 0) sums[A.W] = x;
    }

    if (again) {  // the next step's rows were gathered before these stores
      gather(next);
      // waited for here, so that the other path's wait counts stay exact
#pragma unroll
      for (int k = 0; k < NI; ++k) asm volatile("" : "+v"(next.Gr[k]), "+v"(next.Gw[k]));
    }
  }
};

template <int COLS>
__global__ __launch_bounds__(2 * kWave) void scan_bwd8_kernel(Bwd8Args A) {
  __shared__ __align__(16) Lds8<COLS> sh;
  using S = Scan8<COLS>;
  // XCD-aware numbering as in the forward: every tile of a memory on one XCD
  const int x = blockIdx.x & 7, rest = blockIdx.x >> 3;
  const int tile = rest % A.ntiles, mem = (rest / A.ntiles) * 8 + x;
  if (mem >= A.n_mem) return;  // whole workgroup leaves together
  const int64_t T = A.T, Tp = padded_steps(T);
  const int64_t nchunks = Tp / kChunk;
  const int lane = lane_id(), wave = threadIdx.x / kWave;

  if (wave == 1) {
    // loader: chunks 0 and 1 before the walk starts, then chunk c + 2 while
    // the other wavefront walks chunk c
    const uint8_t* recs = reinterpret_cast<const uint8_t*>(A.rec + (int64_t)mem * Tp);
    auto load = [&](int64_t c) __attribute__((always_inline)) {
      if (c >= nchunks) return;
      constexpr int kPieces = (int)(sizeof(Record) * kChunk / 16);
      const uint8_t* src = recs + c * (int64_t)(sizeof(Record) * kChunk);
      uint8_t* dst = reinterpret_cast<uint8_t*>(&sh.rec[c % kRing][0]);
#pragma unroll
      for (int i = 0; i < (kPieces + kWave - 1) / kWave; ++i)
        if (i * kWave + lane < kPieces)
          __builtin_amdgcn_global_load_lds((const void*)(src + (i * kWave + lane) * 16),
                                           (void*)(dst + i * kWave * 16), 16, 0, 0);
      // v, then dout: kChunk steps of COLS columns; a step before the first: the first
      constexpr int kVec = kChunk * COLS / 4;
      float* vd = &sh.vd[c % kRing][0][0][0];
#pragma unroll
      for (int i = 0; i < (2 * kVec + kWave - 1) / kWave; ++i) {
        const int e = i * kWave + lane, half = e / kVec, s = (e % kVec) / (COLS / 4);
        int64_t t = T - 1 - (c * kChunk + s);
        t = t < 0 ? 0 : t;
        if (e < 2 * kVec)
          __builtin_amdgcn_global_load_lds(
              (const void*)((half ? A.dout : A.v) + ((int64_t)mem * T + t) * A.d_v + tile * COLS +
                            (e % (COLS / 4)) * 4),
              (void*)(vd + i * kWave * 4), 16, 0, 0);
      }
    };
    load(0);
    load(1);
    __builtin_amdgcn_s_waitcnt(0);
    chunk_barrier();
    for (int64_t c = 0; c * kChunk < T; ++c) {
      load(c + 2);
      __builtin_amdgcn_s_waitcnt(0);
      chunk_barrier();
    }
    return;
  }

  const int64_t recs = (int64_t)(A.d_v / 16) * T * (A.W + A.R);
  S s{A, sh};
  s.lr = lane / S::LPR;
  s.lc = lane % S::LPR;
  s.T = T;
  s.lane_off = (uint32_t)s.lc * 16u;
  s.step_rows = (uint32_t)(A.W + A.R);
  s.rec0 = (uint32_t)(tile * (COLS / 16) + s.lc / 4) * (uint32_t)(T * (A.W + A.R)) +
           (uint32_t)((lane & 3) * S::RPI + s.lr);
  // descriptor ranges from ranges.h (checked on the host before the launch)
  s.gres = __builtin_amdgcn_make_buffer_rsrc(
      A.G + (int64_t)mem * A.N * A.d_v + tile * COLS, 0,
      (int)ranges::table_range(A.N, (int64_t)A.d_v * 4, tile, COLS * 4), kBufWord3);
  s.tres = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(A.tape) + (int64_t)mem * recs * 16,
                                             0, (int)ranges::table_range(recs, 16, 0, 16), kBufWord3);
  s.sres = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(A.tape_scale) + (int64_t)mem * recs, 0, (int)recs, kBufWord3);
  float* dv = A.dv + ((int64_t)mem * T + T - 1) * A.d_v + tile * COLS;
  float* sums = A.sums + (((int64_t)mem * T + T - 1) * A.ntiles + tile) * (A.W + 1);
  const int64_t sums_step = (int64_t)A.ntiles * (A.W + 1);

  chunk_barrier();
  typename S::Step even, odd;
  s.issue(even, 0);
  for (int64_t u = 0; u < T; u += 2) {
    s.step(even, odd, u, dv - u * A.d_v, sums - u * sums_step);
    if (u + 1 < T) s.step(odd, even, u + 1, dv - (u + 1) * A.d_v, sums - (u + 1) * sums_step);
    // end of a chunk: its LDS reads are done; the next but one is in
    if ((u + 2) % kChunk == 0 || u + 2 >= T) {
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      chunk_barrier();
    }
  }
}

// dwk = beta * sum over tiles of d(beta k); dalpha = sum; dbeta = sum_j k_j *
// d(beta k_j).  One wavefront per step.
__global__ __launch_bounds__(256) void finish_kernel(Bwd8Args A) {
  const int64_t u = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (u >= (int64_t)A.n_mem * A.T) return;  // whole wavefront leaves together
  const int lane = lane_id(), W = A.W;
  const float* p = A.sums + u * A.ntiles * (W + 1);
  float sbk = 0.0f, sda = 0.0f;
  for (int tl = 0; tl < A.ntiles; ++tl) {
    if (lane < W) sbk += p[tl * (W + 1) + lane];
    sda += p[tl * (W + 1) + W];
  }
  const float kj = lane < W ? A.wk[u * W + lane] : 0.0f;
  if (lane < W) A.dwk[u * W + lane] = A.beta[u] * sbk;
  const float db = wave_sum_f32(lane < W ? kj * sbk : 0.0f);
  if (lane == 0) {
    A.dalpha[u] = sda;
    A.dbeta[u] = db;
  }
}

}  // namespace

size_t scan_backward8_workspace_bytes(int n_mem, int d_v, int64_t T, int W) {
  return (size_t)n_mem * ((size_t)padded_steps(T) * sizeof(Record) +
                          (size_t)T * (size_t)(d_v / 16) * (size_t)(W + 1) * sizeof(float));
}

hipError_t launch_scan_backward8(int B, int H, int64_t N, int d_v, int64_t T, int W, int R,
                                 const int32_t* widx, const float* wk, const int32_t* ridx,
                                 const float* rw, const float* v, const float* alpha,
                                 const float* beta, const int8_t* tape,
                                 const uint8_t* tape_scale, const float* dout, float* G,
                                 float* dv, float* dwk, float* drw, float* dalpha, float* dbeta,
                                 const uint64_t* first, void* ws, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  if (!ranges::tape8_ok(d_v, T, W, R)) return hipErrorInvalidValue;  // checked by the C-ABI layer
  const int n_mem = B * H;
  const int cols = first ? 16 : (d_v < 32 ? d_v : 32);
  const int64_t Tp = padded_steps(T);
  Record* const rec = reinterpret_cast<Record*>(ws);
  Bwd8Args A{n_mem, N,    d_v, T,  W,   R,   widx,   wk,    ridx,  rw,  v,
             alpha, beta, dout, tape, tape_scale, G, dv, dwk, drw, dalpha, dbeta, first, rec,
             reinterpret_cast<float*>(rec + (int64_t)n_mem * Tp), d_v / cols, cols};
  hipLaunchKernelGGL(prepare_kernel, dim3((unsigned)(((int64_t)n_mem * Tp + 3) / 4)), dim3(256), 0,
                     stream, A);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t blocks = (int64_t)((n_mem + 7) / 8) * A.ntiles * 8;
  if (cols == 32)
    hipLaunchKernelGGL(scan_bwd8_kernel<32>, dim3((unsigned)blocks), dim3(2 * kWave), 0, stream, A);
  else
    hipLaunchKernelGGL(scan_bwd8_kernel<16>, dim3((unsigned)blocks), dim3(2 * kWave), 0, stream, A);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(finish_kernel, dim3((unsigned)(((int64_t)n_mem * T + 3) / 4)), dim3(256), 0,
                     stream, A);
  return hipGetLastError();
}

}  // namespace sdm
