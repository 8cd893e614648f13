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
// A whole number times its block's scale is exact in binary32, so the products
// are with the rows' values, as from an fp32 tape.  (The scales multiplying
// sums of products with the whole numbers, up to 127 times the values of a
// block, made sums infinite that are not.)
#include "internal.h"
#include "mx.h"
#include "ranges.h"

namespace sdm {
namespace {

constexpr int kBufWord3 = 0x00020000;  // raw buffer access, gfx9 family
constexpr uint32_t kOffNone = ranges::kOffNone;

constexpr int kChunk = 8;  // records per LDS chunk
constexpr int kRing = 3;

// A step's record.  Row entries are transposed for the tile width in use (COLS
// columns, RPI = 256 / COLS rows per wave instruction, NI = COLS / 4
// instructions for 64): entry lr * NI + k is row slot k * RPI + lr, so a lane
// reads its rows contiguously.  Offsets are multiples of 64
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

// A set of rows as bits: three bits of one of kSetWords words per row (word
// and bits from two multiplicative hashes).  Of 128 rows in the set, an absent
// row is found about once in 3000.
constexpr int kSetWords = 512;
__device__ __forceinline__ uint32_t set_word(uint32_t row) { return (row * 2654435761u) >> 23; }
__device__ __forceinline__ uint32_t set_bits(uint32_t row) {
  const uint32_t h = row * 0x85EBCA77u;
  return (1u << (h >> 27)) | (1u << ((h >> 22) & 31u)) | (1u << ((h >> 17) & 31u));
}

__global__ __launch_bounds__(256) void prepare_kernel(Bwd8Args A) {
  __shared__ uint32_t sets[4][2][kSetWords];
  const int64_t Tp = padded_steps(A.T);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
  if (unit >= (int64_t)A.n_mem * Tp) return;  // whole wavefront leaves together
  const int64_t mem = unit / Tp, u = unit - mem * Tp, t = A.T - 1 - u;
  const int lane = lane_id(), W = A.W, R = A.R;
  Record& out = A.rec[unit];
  const int rpi = 256 / A.cols, at = (lane % rpi) * (A.cols / 4) + lane / rpi;  // slot in the record
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
  uint32_t w1 = ~0u, r1 = ~0u;  // step t + 1's
  if (u > 0) {
    w1 = row(A.widx, W, step + 1);
    r1 = row(A.ridx, R, step + 1);
  }
  const float wk = lane < W ? A.wk[step * W + lane] : 0.0f;
  const float rw = lane < R ? A.rw[step * R + lane] : 0.0f;
  const uint64_t fw = A.first ? A.first[step * 2] : 0ull, fr = A.first ? A.first[step * 2 + 1] : 0ull;

  // Which rows to look at exactly: write rows in the set of this step's read
  // rows, and any row in the set of the rows of step t + 1.
  uint32_t (&reads)[kSetWords] = sets[wave][0], (&later)[kSetWords] = sets[wave][1];
#pragma unroll
  for (int i = 0; i < 2 * kSetWords / 4 / kWave; ++i)
    reinterpret_cast<uint4*>(reads)[i * kWave + lane] = make_uint4(0, 0, 0, 0);  // both
  wave_sync();
  if (r != ~0u) atomicOr(&reads[set_word(r)], set_bits(r));
  if (w1 != ~0u) atomicOr(&later[set_word(w1)], set_bits(w1));
  if (r1 != ~0u) atomicOr(&later[set_word(r1)], set_bits(r1));
  wave_sync();
  const uint32_t bw = set_bits(w), br = set_bits(r);
  uint64_t match = __ballot(w != ~0u && (reads[set_word(w)] & bw) == bw);
  const uint64_t aw = __ballot(w != ~0u && (later[set_word(w)] & bw) == bw);
  const uint64_t ar = __ballot(r != ~0u && (later[set_word(r)] & br) == br);
  // the read weight that falls on a write row (read rows are distinct)
  float mw = 0.0f;
  for (; match; match &= match - 1) {
    const int l = __builtin_ctzll(match);
    const uint64_t hit = __ballot(r == (uint32_t)__builtin_amdgcn_readlane((int)w, l));
    const float x = __uint_as_float((uint32_t)__builtin_amdgcn_readlane(
        (int)__float_as_uint(rw), hit ? __builtin_ctzll(hit) : 0));
    if (lane == l && hit) mw = x;
  }
  // rows shared with step t + 1
  bool shared = false;
  for (uint64_t m = aw; m && !shared; m &= m - 1) {
    const uint32_t s = (uint32_t)__builtin_amdgcn_readlane((int)w, __builtin_ctzll(m));
    shared = __ballot(w1 == s || r1 == s) != 0ull;
  }
  for (uint64_t m = ar; m && !shared; m &= m - 1) {
    const uint32_t s = (uint32_t)__builtin_amdgcn_readlane((int)r, __builtin_ctzll(m));
    shared = __ballot(w1 == s || r1 == s) != 0ull;
  }
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
  const int nb = A.d_v / 16;
  const int64_t S = A.T * (W + R), rec = mem * nb * S + t * (W + R) + W + lane;
  const float* d = A.dout + step * A.d_v;
  float dr = 0.0f;
#pragma unroll 2
  for (int b = 0; b < nb; ++b) {
    u32x4 q = {0u, 0u, 0u, 0u};
    uint32_t scale = 0;
    if (r != ~0u) {  // lanes past R among them: nothing is read there
      q = *reinterpret_cast<const u32x4*>(A.tape + (rec + b * S) * 16);
      scale = A.tape_scale[rec + b * S];
    }
    const uint32_t c[4] = {q.x, q.y, q.z, q.w};
    const float sc = scale_value(scale);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[4];
      int8_unpack4(c[i], x);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fmaf(d[b * 16 + 4 * i + e], x[e] * sc, s);
    }
    dr += s;
  }
  if (lane < R) A.drw[step * R + lane] = dr;
}

// ---------------------------------------------------------------- scan

template <int COLS, int NC>
struct Lds8 {
  Record rec[kRing][kChunk];
  float vd[kRing][2][kChunk][NC * COLS];  // the workgroup's columns of v and dout
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

template <int COLS, int NC>
struct Scan8 {
  static constexpr int LPR = COLS / 4, RPI = kWave / LPR, NI = 64 / RPI;
  static_assert(NI == LPR, "lane lc of a row ends with the sums of instruction lc's row");

  // A step in flight: its offsets, its rows of G and its pre-write records.
  struct Step {
    uint32_t wo[NI], ro[NI];
    u32x4 Gw[NI], Gr[NI];
    u32x4 codes;     // 16 columns: see issue(); 8: a word per instruction
    uint8_t scale[COLS == 16 ? 1 : NI];  // as loaded: widened at its use, so that nothing waits before
  };

  const Bwd8Args& A;
  Lds8<COLS, NC>& sh;
  __amdgpu_buffer_rsrc_t gres, tres, sres;
  uint32_t lane_off, rec0, step_rows;
  uint32_t word;  // 8 columns: byte offset of the lane's four codes in a record
  int lr, lc, col0, T;

  __device__ __forceinline__ const Record& record(int u) const {
    return sh.rec[(uint32_t)u / kChunk % kRing][u % kChunk];
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

  __device__ __forceinline__ void issue(Step& s, int u) const {
    const Record& r = record(u);
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      s.wo[k] = r.wofs[lr * NI + k];
      s.ro[k] = r.rofs[lr * NI + k];
    }
    gather(s);
    const uint32_t rec = rec0 + (uint32_t)(T - 1 - u) * step_rows;
    if constexpr (COLS == 16) {
      // the whole tape record (16 code bytes, a scale) of slot lc * RPI + lr:
      // one load of each for 64 rows; the quads exchange the codes' words later
      const bool none = r.wofs[lr * NI + lc] >= kOffNone;
      const uint32_t at = rec + (uint32_t)(lc * RPI + lr);
      s.codes = __builtin_amdgcn_raw_buffer_load_b128(tres, none ? kOffNone : at * 16u, 0, 0);
      s.scale[0] = __builtin_amdgcn_raw_buffer_load_b8(sres, none ? kOffNone : at, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < NI; ++k) {
        const bool none = s.wo[k] >= kOffNone;
        const uint32_t at = rec + (uint32_t)(k * RPI + lr);
        s.codes[k] = __builtin_amdgcn_raw_buffer_load_b32(tres, none ? kOffNone : at * 16u + word, 0, 0);
        s.scale[k] = __builtin_amdgcn_raw_buffer_load_b8(sres, none ? kOffNone : at, 0, 0);
      }
    }
  }

  // Step u, with step u + 1's loads going out first.
  __device__ __forceinline__ void step(Step& s, Step& next, int u, float* dv, float* sums) const {
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
    const int ring = (uint32_t)u / kChunk % kRing, at = u % kChunk;
    const f32x4 vv = *reinterpret_cast<const f32x4*>(&sh.vd[ring][0][at][col0 + lc * 4]);
    const f32x4 dd = *reinterpret_cast<const f32x4*>(&sh.vd[ring][1][at][col0 + lc * 4]);

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
    // word k: this lane's four codes of slot k * RPI + lr, sc[k] their scale
    uint32_t w[4] = {s.codes.x, s.codes.y, s.codes.z, s.codes.w};
    float sc[NI];
    if constexpr (COLS == 16) {
      quad_transpose(w);
      const uint32_t scale = __float_as_uint(scale_value(s.scale[0]));
      sc[0] = __uint_as_float(dpp_mov<0x00>(scale));
      sc[1] = __uint_as_float(dpp_mov<0x55>(scale));
      sc[2] = __uint_as_float(dpp_mov<0xAA>(scale));
      sc[3] = __uint_as_float(dpp_mov<0xFF>(scale));
    } else {
#pragma unroll
      for (int k = 0; k < NI; ++k) sc[k] = scale_value(s.scale[k]);
    }
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      float p[4];
      int8_unpack4(w[k], p);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] *= sc[k];
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
      da = fmaf(keep, gp, da);
      dbk[k] = g.x * (vv.x - a * p[0]) + g.y * (vv.y - a * p[1]) + g.z * (vv.z - a * p[2]) +
               g.w * (vv.w - a * p[3]);
      const float c = a * keep;
      s.Gw[k] = as_u4(f32x4{c * g.x, c * g.y, c * g.z, c * g.w});
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
    float f = fold<0>(dbk[0], dbk[1]);
    if constexpr (NI == 4) f = fold<1>(f, fold<0>(dbk[2], dbk[3]));
    const int j = lc * RPI + lr;
    if (j < A.W) sums[j] = f;
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
      x += __uint_as_float(dpp_row_ror4(__float_as_uint(x)));
      if constexpr (LPR == 2) x += __uint_as_float(dpp_mov<0x122>(__float_as_uint(x)));  // ror 2
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

template <int COLS, int NC>
__global__ __launch_bounds__((NC + 1) * kWave) void scan_bwd8_kernel(Bwd8Args A) {
  __shared__ __align__(16) Lds8<COLS, NC> sh;
  using S = Scan8<COLS, NC>;
  // XCD-aware numbering as in the forward: every tile of a memory on one XCD
  const int x = blockIdx.x & 7, rest = blockIdx.x >> 3;
  const int groups = A.ntiles / NC;
  const int tile0 = (rest % groups) * NC, mem = (rest / groups) * 8 + x;
  if (mem >= A.n_mem) return;  // whole workgroup leaves together
  const int T = (int)A.T, Tp = (int)padded_steps(T);  // below 2^26 (checked on the host)
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

  if (wave == NC) {
    // loader: chunks 0 and 1 before the walk starts, then chunk c + 2 while
    // the others walk chunk c
    const uint8_t* recs = reinterpret_cast<const uint8_t*>(A.rec + (int64_t)mem * Tp);
    auto load = [&](int c) __attribute__((always_inline)) {
      if (c * kChunk >= Tp) return;
      constexpr int kPieces = (int)(sizeof(Record) * kChunk / 16);
      const uint8_t* src = recs + c * (int64_t)(sizeof(Record) * kChunk);
      uint8_t* dst = reinterpret_cast<uint8_t*>(&sh.rec[c % kRing][0]);
#pragma unroll
      for (int i = 0; i < (kPieces + kWave - 1) / kWave; ++i)
        if (i * kWave + lane < kPieces)
          __builtin_amdgcn_global_load_lds((const void*)(src + (i * kWave + lane) * 16),
                                           (void*)(dst + i * kWave * 16), 16, 0, 0);
      // v, then dout: kChunk steps of the columns; a step before the first: the first
      constexpr int kPer = NC * COLS / 4, kVec = kChunk * kPer;
      float* vd = &sh.vd[c % kRing][0][0][0];
#pragma unroll
      for (int i = 0; i < (2 * kVec + kWave - 1) / kWave; ++i) {
        const int e = i * kWave + lane, half = e / kVec, s = (e % kVec) / kPer;
        int t = T - 1 - (c * kChunk + s);
        t = t < 0 ? 0 : t;
        if (e < 2 * kVec)
          __builtin_amdgcn_global_load_lds(
              (const void*)((half ? A.dout : A.v) + ((int64_t)mem * T + t) * A.d_v + tile0 * COLS +
                            (e % kPer) * 4),
              (void*)(vd + i * kWave * 4), 16, 0, 0);
      }
    };
    load(0);
    load(1);
    __builtin_amdgcn_s_waitcnt(0);
    chunk_barrier();
    for (int u = 0; u < T; u += 2) {
      if (u % kChunk == 0) load(u / kChunk + 2);
      if ((u + 2) % kChunk == 0) __builtin_amdgcn_s_waitcnt(0);
      chunk_barrier();
    }
    // (a chunk still on its way at the end lands before the wavefront ends)
    __builtin_amdgcn_s_waitcnt(0);
    return;
  }

  const int tile = tile0 + wave;
  const int64_t recs = (int64_t)(A.d_v / 16) * T * (A.W + A.R);
  S s{A, sh};
  s.lr = lane / S::LPR;
  s.lc = lane % S::LPR;
  s.col0 = wave * COLS;
  s.word = (uint32_t)(tile * COLS % 16 + s.lc * 4);
  s.T = T;
  s.lane_off = (uint32_t)s.lc * 16u;
  s.step_rows = (uint32_t)(A.W + A.R);
  s.rec0 = (uint32_t)(tile * COLS / 16) * (uint32_t)((int64_t)T * (A.W + A.R));
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
  // As many stores as a step makes after its loads, to offsets past the range
  // (dropped; distinct, or they would be merged): the compiler's wait counts at
  // the loop's head are the tighter of the two ways into it.
#pragma unroll
  for (int i = 0; i < 2 * S::NI; ++i)
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{0u, 0u, 0u, 0u}, s.gres,
                                           kOffNone + (uint32_t)i * 16u, 0, 0);
  const int64_t dv_step = -(int64_t)A.d_v;
  int u = 0;
  for (; u + 1 < T; u += 2, dv += 2 * dv_step, sums -= 2 * sums_step) {
    s.step(even, odd, u, dv, sums);
    s.step(odd, even, u + 1, dv + dv_step, sums - sums_step);
    // Every two steps: keeps the two halves of a cache line of G close in time
    // and, at a chunk's end (its LDS reads are done), the ring in step.
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    chunk_barrier();
  }
  if (u < T) {
    s.step(even, odd, u, dv, sums);
    chunk_barrier();
  }
}

// dwk = beta * sum over tiles of d(beta k); dalpha = sum; dbeta = sum_j k_j *
// d(beta k_j).  One wavefront per step.
__global__ __launch_bounds__(256) void finish_kernel(Bwd8Args A) {
  const int64_t u = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (u >= (int64_t)A.n_mem * A.T) return;  // whole wavefront leaves together
  const int lane = lane_id(), W = A.W;
  const float* p = A.sums + u * A.ntiles * (W + 1);
  const int at = lane < W ? lane : W;  // lanes past W: dalpha's word again
  float sbk = 0.0f, sda = 0.0f;
#pragma unroll 4
  for (int tl = 0; tl < A.ntiles; ++tl) {
    sbk += p[tl * (W + 1) + at];
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

namespace {

// Columns of a wavefront's tile.  Few memories: the scan goes at the pace of
// one wavefront's instructions for a step, so with room for 8-column tiles on
// a compute unit each (half the rows' instructions, twice the wavefronts) they
// are taken.  With 8 and 16 columns, us: 4 memories x 301 steps (d_v 64) 178 and
// 268; 512 steps at d_v 128, dense and sparse, 16 memories 535 428 and 528 481,
// 24 memories 776 629 and 592 549, 32 memories 878 732 and 653 630.
constexpr int kMostUnits = 256;  // compute units of an undivided GPU
bool few_memories(int n_mem, int d_v, int units) { return (int64_t)n_mem * (d_v / 8) <= units; }
int scan_columns(int n_mem, int d_v) {
  const int cus = compute_units();
  return few_memories(n_mem, d_v, cus < kMostUnits ? cus : kMostUnits) ? 8 : 16;
}

}  // namespace

// (for the narrower tiles wherever some GPU would take them: the size is the
// same whichever GPU is current)
size_t scan_backward8_workspace_bytes(int n_mem, int d_v, int64_t T, int W) {
  const int tiles = d_v / (few_memories(n_mem, d_v, kMostUnits) ? 8 : 16);
  return (size_t)n_mem * ((size_t)padded_steps(T) * sizeof(Record) +
                          (size_t)T * (size_t)tiles * (size_t)(W + 1) * sizeof(float));
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
  const int cols = scan_columns(n_mem, d_v);
  const int64_t Tp = padded_steps(T);
  Record* const rec = reinterpret_cast<Record*>(ws);
  Bwd8Args A{n_mem, N,    d_v, T,  W,   R,   widx,   wk,    ridx,  rw,  v,
             alpha, beta, dout, tape, tape_scale, G, dv, dwk, drw, dalpha, dbeta, first, rec,
             reinterpret_cast<float*>(rec + (int64_t)n_mem * Tp), d_v / cols, cols};
  hipLaunchKernelGGL(prepare_kernel, dim3((unsigned)(((int64_t)n_mem * Tp + 3) / 4)), dim3(256), 0,
                     stream, A);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Many memories: the two 16-column halves of each cache line of G go to one
  // workgroup, in step (64 memories: 1.71 against 2.12 ms in the sparse mode of
  // 1024 steps; 16 memories, the chip not filled: 2.15 against 1.90).
  const int nc = cols == 16 && A.ntiles > 1 && (int64_t)n_mem * (A.ntiles / 2) >= compute_units() ? 2 : 1;
  const dim3 blocks((unsigned)((int64_t)((n_mem + 7) / 8) * (A.ntiles / nc) * 8));
  if (nc == 2)
    hipLaunchKernelGGL((scan_bwd8_kernel<16, 2>), blocks, dim3(3 * kWave), 0, stream, A);
  else if (cols == 16)
    hipLaunchKernelGGL((scan_bwd8_kernel<16, 1>), blocks, dim3(2 * kWave), 0, stream, A);
  else
    hipLaunchKernelGGL((scan_bwd8_kernel<8, 1>), blocks, dim3(2 * kWave), 0, stream, A);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(finish_kernel, dim3((unsigned)(((int64_t)n_mem * T + 3) / 4)), dim3(256), 0,
                     stream, A);
  return hipGetLastError();
}

}  // namespace sdm
