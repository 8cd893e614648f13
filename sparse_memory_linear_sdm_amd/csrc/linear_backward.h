// Reverse pass of the dense recurrence with a decay for each head, in the
// forward's chunks (linear_scan.h), last to first.  With S the state before a
// chunk (from the tape), G the gradient of the state behind it, C its last
// step, L_t the sum of g through step t, D_ts = exp(L_t - L_s) for s <= t and
// 0 above:
//   dq_t = exp(L_t) S do_t         + sum over s of (do_t . v_s) D_ts k_s
//   dk_s = exp(L_C - L_s) G v_s    + sum over t of (do_t . v_s) D_ts q_t
//   dv_s = exp(L_C - L_s) G^T k_s  + sum over t of (q_t . k_s) D_ts do_t
//   G'   = exp(L_C) G              + sum over t of exp(L_t) q_t do_t^T
// A step's decay scales every path from a step before it to one at or after
// it, so its gradient is the sum of those paths:
//   dg_t = sum over i >= t > j of W_ij, W_ij = (q_i . k_j)(do_i . v_j) D_ij
//        + sum over i >= t of e_i      e_i = exp(L_i) q_i . S do_i
//        + sum over j < t of f_j       f_j = exp(L_C - L_j) k_j . G v_j
//        + exp(L_C) <S, G>
// No difference of sums is taken: a step that forgets almost everything has a
// small gradient beside large W on either side.  In 16 x 16 tiles of W, the
// first line is a part of t's own tile, rows from t on of the tiles left of it,
// columns before t of those below it, and whole tiles left and below.
//
// One workgroup walks a memory's chunks (or a segment's).  G is kept twice in
// its accumulators, by rows of k and by rows of v: it enters products along
// either index, and an accumulator tile is an operand along its rows.  Each
// wavefront holds 16 columns of both, so there are eight where a head is 128
// wide: G, S and the loads ahead then fit in registers.
//
// Bound by a chunk's phases like the scan, with three times its products: 64
// memories x 2048 steps of 128 x 128 bf16 in four segments, 25 us for the
// segments' states and 141-149 for this pass (18 us a chunk of 64 steps; counted:
// LDS active 50% of the time, vector arithmetic 45%, matrix cores 26%, memory 2.5
// TB/s); fp32 50 + 279 us.
#pragma once
#include "dense.h"
#include "linear_tile.h"

namespace sdm {
namespace lin {

// The sum over lanes l, l ^ 16, l ^ 32 and l ^ 48.
__device__ __forceinline__ float over_quarters(float x) {
  x += __uint_as_float(lane_xor(__float_as_uint(x), 16));
  return x + __uint_as_float(lane_xor(__float_as_uint(x), 32));
}

template <int DK, int DV>
struct BackwardShape {
  static constexpr int kWaves = DK == 128 || DV == 128 ? 8 : 4;
  static constexpr int kThreads = kWaves * kWave;
};

template <class T, int DK, int DV>
__global__ __launch_bounds__((BackwardShape<DK, DV>::kThreads)) void linear_backward_kernel(
    LinearArgs A) {
  typedef Tile<T> X;
  typedef typename X::Frag Frag;
  constexpr int C = X::kChunk;
  constexpr int NW = BackwardShape<DK, DV>::kWaves, NT = NW * kWave;
  typedef Block<T, DK, NT> BlockK;
  typedef Block<T, DV, NT> BlockV;
  typedef Pairs<T> P;
  constexpr int kTT = C / 16, kKT = DK / 16, kVT = DV / 16;
  static_assert(kKT <= NW && kVT <= NW, "one column tile a wavefront");
  __shared__ __align__(16) T sq[BlockK::kSize];
  __shared__ __align__(16) T sk[BlockK::kSize];
  __shared__ __align__(16) T sv[BlockV::kSize];
  __shared__ __align__(16) T so[BlockV::kSize];  // dout
  __shared__ __align__(16) T sp[P::kParts * P::kSize];   // (q_t . k_s) D_ts
  __shared__ __align__(16) T sdp[P::kParts * P::kSize];  // (do_t . v_s) D_ts
  __shared__ Decays<C> sd[2];
  // what dg is summed from, for this chunk and the one before it
  struct Paths {
    // sums of W over the rows and columns of its tiles; row[tile of t][t]: the sum
    // of W_ij, i >= t > j, inside t's tile
    float row[kTT][C], col[kTT][C];
    float e[kKT][C], f[kKT][C];        // by wavefronts
    float x[kKT];                      // exp(L_C) <S, G>
  };
  __shared__ Paths paths[2];

  const int lane = lane_id(), col = lane & 15, g4 = 4 * (lane >> 4);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t pid = xcd_contiguous(blockIdx.x, gridDim.x);
  const int bh = (int)(pid / (uint32_t)A.nseg), seg = (int)(pid % (uint32_t)A.nseg);
  const int c_first = seg * A.seg_chunks;
  const int c_end = c_first + A.seg_chunks < A.nchunk ? c_first + A.seg_chunks : A.nchunk;
  const int64_t key_row = (int64_t)(bh / A.share) * A.T, row = (int64_t)bh * A.T;
  const T* gq = (const T*)A.q + key_row * DK;
  const T* gk = (const T*)A.k + key_row * DK;
  const T* gv = (const T*)A.v + row * DV;
  const T* go = (const T*)A.dout + row * DV;
  const float* gg = A.g + row;
  // this wavefront's columns of k and of v
  const bool has_k = kKT == NW || w < kKT, has_v = kVT == NW || w < kVT;
  const int k0 = w * 16, v0 = w * 16;

  f32x4 Gk[kKT];  // rows of k, columns v0 .. v0 + 15
  f32x4 Gv[kVT];  // rows of v, columns k0 .. k0 + 15
  auto add_state = [&](const float* from, float decay) {  // G = decay G + from
    const __amdgpu_buffer_rsrc_t b = buffer(from, DK * DV * 4);
    if (has_v) {
#pragma unroll
      for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          Gk[kt][i] = Gk[kt][i] * decay +
                      buffer_float(b, (g4 * DV + v0 + col) * 4, (kt * 16 + i) * DV * 4);
    }
    if (has_k) {
#pragma unroll
      for (int vt = 0; vt < kVT; ++vt)
        Gv[vt] = Gv[vt] * decay +
                 __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                               b, ((k0 + col) * DV + g4 + vt * 16) * 4, 0, 0));
    }
  };
#pragma unroll
  for (int kt = 0; kt < kKT; ++kt) Gk[kt] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int vt = 0; vt < kVT; ++vt) Gv[vt] = f32x4{0, 0, 0, 0};
  BlockK bq, bk;
  BlockV bv, bo;
  // steps of chunk c, 0 before the first one
  auto rows_of = [&](int c) {
    const int64_t left = A.T - (int64_t)c * C;
    return c < c_first ? 0 : left < C ? (int)left : C;
  };
  auto load = [&](int c) {
    const int64_t t0 = (int64_t)c * C;
    const int valid = rows_of(c);
    bq.load(gq + t0 * DK, valid);
    bk.load(gk + t0 * DK, valid);
    bv.load(gv + t0 * DV, valid);
    bo.load(go + t0 * DV, valid);
  };
  auto g_of = [&](int c) {  // of step `lane` of chunk c
    return __builtin_bit_cast(
        float, __builtin_amdgcn_raw_buffer_load_b32(
                   buffer(gg + (int64_t)c * C, (uint32_t)rows_of(c) * 4), lane * 4, 0, 0));
  };
  // the state before the chunk, rows k0 .. k0 + 15, as operands along v
  f32x4 S[kVT];
  auto load_state = [&](int c) {
    const __amdgpu_buffer_rsrc_t b = buffer(A.tape + ((int64_t)bh * A.nchunk + c) * DK * DV,
                                            c < c_first ? 0 : DK * DV * 4);
#pragma unroll
    for (int vt = 0; vt < kVT; ++vt)
      S[vt] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                            b, ((k0 + col) * DV + g4 + vt * 16) * 4, 0, 0));
  };
  // dg of chunk c, by one wavefront
  auto gate = [&](int c, float g) {
    const Paths& p = paths[c & 1];
    const int tile = lane >> 4;
    double e = 0.0, f = 0.0, x = 0.0, down = 0.0, left[kTT - 1] = {};
    if (lane < C) {
      x = (double)p.row[tile][lane];
#pragma unroll
      for (int i = 0; i < kTT; ++i) {
        if (i < kTT - 1 && i < tile) left[i] = (double)p.row[i][lane];
        if (i > tile) down += (double)p.col[i][lane];
      }
#pragma unroll
      for (int i = 0; i < kKT; ++i) {
        e += (double)p.e[i][lane];
        f += (double)p.f[i][lane];
        x += (double)p.x[i];
      }
    }
    // steps from this one on, and before it, in its tile; then whole tiles
    e = row_sums_up(e);
    f = row_sums_down(f);
#pragma unroll
    for (int i = 0; i < kTT - 1; ++i) {
      left[i] = row_sums_up(left[i]);
      x += left[i];
    }
    x += e + row_shr<1>(f) + row_shr<1>(row_sums_down(down));
#pragma unroll
    for (int r = 0; r < kTT; ++r) {
      const double e_tile = lane_value(e, r * 16), f_tile = lane_value(f, r * 16 + 15);
      x += r > tile ? e_tile : r < tile ? f_tile : 0.0;
#pragma unroll
      for (int i = 0; i + 1 < r; ++i) {
        const double w_tile = lane_value(left[i], r * 16);
        x += i < tile && tile < r ? w_tile : 0.0;
      }
    }
    // a step that forgets everything has no path across it: exactly 0
    const float dg = g <= -128.0f ? 0.0f : (float)x;
    __builtin_amdgcn_raw_buffer_store_b32(
        __float_as_uint(dg), buffer(A.dg + row + (int64_t)c * C, (uint32_t)rows_of(c) * 4),
        lane * 4, 0, 0);
  };

  // g runs one chunk further ahead than the blocks, its sums come first
  float g_now = g_of(c_end - 1), g_next = g_of(c_end - 2), g_last = 0.0f;
  load(c_end - 1);
  if (has_k) load_state(c_end - 1);
  {
    const float* states = A.seg_state + (int64_t)bh * A.nseg * DK * DV;
    if (A.nseg == 1) {
      add_state(A.S + (int64_t)bh * DK * DV, 0.0f);
    } else if (A.nseg > kOwnSegments) {
      add_state(states + (int64_t)seg * DK * DV, 0.0f);
    } else {
      add_state(states, 0.0f);  // the call's gradient
      for (int i = A.nseg - 1; i > seg; --i)
        add_state(states + (int64_t)i * DK * DV, pow2((float)A.seg_log[(int64_t)bh * A.nseg + i]));
    }
  }
  if (w == NW - 1) scan_decays<C>(log2_decay(g_now), sd[(c_end - 1) & 1]);
  arrive(Gk);
  arrive(Gv);

  for (int c = c_end - 1; c >= c_first; --c) {
    const Decays<C>& d = sd[c & 1];
    Paths& path = paths[c & 1];
    const int64_t t0 = (int64_t)c * C;
    const int valid = rows_of(c);
    bq.store(sq);
    bk.store(sk);
    bv.store(sv);
    bo.store(so);
    __syncthreads();
    const float g_ahead = g_of(c - 2);
    load(c - 1);
    if (w == NW / 2 && c + 1 < c_end) gate(c + 1, g_last);
    // ---- pairs of steps: P, dP and the sums of W
    constexpr int kUnits = kTT == 4 ? 12 : 4;  // tiles that a product below reads
#pragma unroll
    for (int u0 = 0; u0 < kUnits; u0 += NW) {
      const int u = u0 + w;
      if (u0 + NW > kUnits && u >= kUnits) continue;
      const int tt = u < 4 ? u >> 1 : 2 + ((u - 4) >> 2), st = u < 4 ? u & 1 : (u - 4) & 3;
      f32x4 p = {0, 0, 0, 0}, dp = {0, 0, 0, 0};
      const int t = tt * 16 + col, s = st * 16 + g4;
      schedule_end();
#pragma unroll
      for (int kb = 0; kb < DK / 32; ++kb)
        p = X::mma(X::template rows<DK>(sk, st * 16, kb * 32),
                   X::template rows<DK>(sq, tt * 16, kb * 32), p);
#pragma unroll
      for (int vb = 0; vb < DV / 32; ++vb)
        dp = X::mma(X::template rows<DV>(sv, st * 16, vb * 32),
                    X::template rows<DV>(so, tt * 16, vb * 32), dp);
      schedule_reads<6 * X::kRowReads>();  // three pairs ahead
#pragma unroll
      for (int i = 0; i < (DK + DV) / 32; ++i) {
        schedule_reads<2 * X::kRowReads>();
        schedule_products<X::kProducts>();
      }
      schedule_end();
      const f32x4 decay = decay_between<C>(d, t, s);
      const f32x4 raw = dp;
      p = decayed(p, decay, t, s);
      dp = decayed(dp, decay, t, s);
      // W's sums over rows t .. 15 of the tile by columns, over its columns by rows;
      // in the diagonal tile the former over the columns before t
      float by_row = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float W = s + j < t ? p[j] * raw[j] : 0.0f;
        const float down = row_sums_up(W);
        if (col == 0) path.col[tt][s + j] = down;
        by_row += tt != st ? W : s + j < t ? down : 0.0f;
      }
      by_row = over_quarters(by_row);
      if (lane < 16) path.row[st][t] = by_row;
      P::store4(sp, t, s, p);
      P::store4(sdp, t, s, dp);
    }
    if (w == NW - 1) scan_decays<C>(log2_decay(g_next), sd[(c - 1) & 1]);
    __syncthreads();

    // ---- the gradients, transposed (a lane holds four consecutive values of one
    // step): the state's part, then the pairs'.  Then G before the chunk.
    const float whole = d.whole;
    if (has_k) {
      const bool shared = A.share > 1;
      const int64_t at0 = (row + t0) * DK;
      const uint32_t bytes = valid * DK * (shared ? 4 : (int)sizeof(T));
      const __amdgpu_buffer_rsrc_t
          out_q = buffer(shared ? (void*)(A.dq_part + at0) : (void*)((T*)A.dq + at0), bytes),
          out_k = buffer(shared ? (void*)(A.dk_part + at0) : (void*)((T*)A.dk + at0), bytes);
      f32x4 a[kTT];
      auto store_rows = [&](__amdgpu_buffer_rsrc_t out) {
        if (shared) {
#pragma unroll
          for (int i = 0; i < kTT; ++i)
            Tile<float>::store4(out, (i * 16 + col) * DK + k0 + g4, a[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kTT; ++i) X::store4(out, (i * 16 + col) * DK + k0 + g4, a[i]);
        }
      };
      float x = 0.0f;
      // dq.  S and G enter dg with fp32's precision, in parts
#pragma unroll
      for (int i = 0; i < kTT; ++i) a[i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int vb = 0; vb < DV / 32; ++vb) {
        const f32x8 s = Tile<float>::pack(S[2 * vb], S[2 * vb + 1]);
        const f32x8 G = Tile<float>::pack(Gv[2 * vb], Gv[2 * vb + 1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) x += s[j] * G[j];
        Frag part[X::kParts];
        X::split(s, part);
        Frag o[kTT];
#pragma unroll
        for (int i = 0; i < kTT; ++i) o[i] = X::template rows<DV>(so, i * 16, vb * 32);
#pragma unroll
        for (int p = 0; p < X::kParts; ++p)
#pragma unroll
          for (int i = 0; i < kTT; ++i) a[i] = X::mma(part[p], o[i], a[i]);
      }
      load_state(c - 1);
      x = wave_sum_f32(x);
      if (lane == 0) path.x[w] = x * whole;
      {
        Frag kc[C / 32];
#pragma unroll
        for (int b = 0; b < C / 32; ++b) kc[b] = X::template cols<DK>(sk, b * 32, k0);
#pragma unroll
        for (int i = 0; i < kTT; ++i) {
          const int t = i * 16 + col;
          a[i] *= d.into[t];
          const f32x4 q = X::load4(sq + X::template at<DK>(t, k0 + g4));
          const float e = over_quarters((q[0] * a[i][0] + q[1] * a[i][1]) +
                                        (q[2] * a[i][2] + q[3] * a[i][3]));
          if (lane < 16) path.e[w][t] = e;
#pragma unroll
          for (int b = 0; b <= i / 2; ++b)
#pragma unroll
            for (int j = 0; j < P::kParts; ++j)
              a[i] = X::mma(kc[b], P::rows(sdp, j, i * 16, b * 32), a[i]);
        }
        store_rows(out_q);
      }
      // dk
#pragma unroll
      for (int i = 0; i < kTT; ++i) a[i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int vb = 0; vb < DV / 32; ++vb) {
        Frag part[X::kParts];
        X::split(Tile<float>::pack(Gv[2 * vb], Gv[2 * vb + 1]), part);
        Frag v[kTT];
#pragma unroll
        for (int i = 0; i < kTT; ++i) v[i] = X::template rows<DV>(sv, i * 16, vb * 32);
#pragma unroll
        for (int p = 0; p < X::kParts; ++p)
#pragma unroll
          for (int i = 0; i < kTT; ++i) a[i] = X::mma(part[p], v[i], a[i]);
      }
      Frag qc[C / 32];
#pragma unroll
      for (int b = 0; b < C / 32; ++b) qc[b] = X::template cols<DK>(sq, b * 32, k0);
#pragma unroll
      for (int i = 0; i < kTT; ++i) {
        const int t = i * 16 + col;
        a[i] *= d.onto[t];
        const f32x4 k = X::load4(sk + X::template at<DK>(t, k0 + g4));
        const float f = over_quarters((k[0] * a[i][0] + k[1] * a[i][1]) +
                                      (k[2] * a[i][2] + k[3] * a[i][3]));
        if (lane < 16) path.f[w][t] = f;
#pragma unroll
        for (int b = i / 2; b < C / 32; ++b)
#pragma unroll
          for (int j = 0; j < P::kParts; ++j)
            a[i] = X::mma(qc[b], P::cols(sdp, j, b * 32, i * 16), a[i]);
      }
      store_rows(out_k);
      Frag part[C / 32][X::kParts];
#pragma unroll
      for (int b = 0; b < C / 32; ++b)
        X::split(X::widen(qc[b]) *
                     Tile<float>::pack(*reinterpret_cast<const f32x4*>(d.into + b * 32 + g4),
                                       *reinterpret_cast<const f32x4*>(d.into + b * 32 + 16 + g4)),
                 part[b]);
      schedule_end();
#pragma unroll
      for (int vt = 0; vt < kVT; ++vt) {
        Gv[vt] *= whole;
#pragma unroll
        for (int b = 0; b < C / 32; ++b) {
          const Frag o = X::template cols<DV>(so, b * 32, vt * 16);
#pragma unroll
          for (int p = 0; p < X::kParts; ++p) Gv[vt] = X::mma(o, part[b][p], Gv[vt]);
        }
      }
      schedule_reads<4 * X::kColReads>();  // four fragments ahead
#pragma unroll
      for (int j = 0; j < kVT * (C / 32); ++j) {
        schedule_reads<X::kColReads>();
        schedule_products<X::kParts * X::kProducts>();
      }
      schedule_end();
    }
    if (has_v) {
      const __amdgpu_buffer_rsrc_t out_v =
          buffer((T*)A.dv + (row + t0) * DV, (uint32_t)(valid * DV * (int)sizeof(T)));
      f32x4 a[kTT];
#pragma unroll
      for (int i = 0; i < kTT; ++i) a[i] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kb = 0; kb < DK / 32; ++kb) {
        Frag G[X::kOutParts], k[kTT];
        X::template split<X::kOutParts>(Tile<float>::pack(Gk[2 * kb], Gk[2 * kb + 1]), G);
#pragma unroll
        for (int i = 0; i < kTT; ++i) k[i] = X::template rows<DK>(sk, i * 16, kb * 32);
#pragma unroll
        for (int j = 0; j < X::kOutParts; ++j)
#pragma unroll
          for (int i = 0; i < kTT; ++i) a[i] = X::mma(G[j], k[i], a[i]);
      }
      schedule_reads<2 * kTT * X::kRowReads>();
#pragma unroll
      for (int kb = 0; kb < DK / 32; ++kb) {
        schedule_reads<kTT * X::kRowReads>();
        schedule_products<kTT * X::kOutParts * X::kProducts>();
      }
      schedule_end();
      Frag oc[C / 32];
#pragma unroll
      for (int b = 0; b < C / 32; ++b) oc[b] = X::template cols<DV>(so, b * 32, v0);
#pragma unroll
      for (int i = 0; i < kTT; ++i) {
        a[i] *= d.onto[i * 16 + col];
#pragma unroll
        for (int b = i / 2; b < C / 32; ++b)
#pragma unroll
          for (int j = 0; j < P::kParts; ++j)
            a[i] = X::mma(oc[b], P::cols(sp, j, b * 32, i * 16), a[i]);
        X::store4(out_v, (i * 16 + col) * DV + v0 + g4, a[i]);
      }
      Frag part[C / 32][X::kParts];
#pragma unroll
      for (int b = 0; b < C / 32; ++b)
        X::split(X::widen(oc[b]) *
                     Tile<float>::pack(*reinterpret_cast<const f32x4*>(d.into + b * 32 + g4),
                                       *reinterpret_cast<const f32x4*>(d.into + b * 32 + 16 + g4)),
                 part[b]);
      schedule_end();
#pragma unroll
      for (int kt = 0; kt < kKT; ++kt) {
        Gk[kt] *= whole;
#pragma unroll
        for (int b = 0; b < C / 32; ++b) {
          const Frag q = X::template cols<DK>(sq, b * 32, kt * 16);
#pragma unroll
          for (int p = 0; p < X::kParts; ++p) Gk[kt] = X::mma(q, part[b][p], Gk[kt]);
        }
      }
      schedule_reads<4 * X::kColReads>();
#pragma unroll
      for (int j = 0; j < kKT * (C / 32); ++j) {
        schedule_reads<X::kColReads>();
        schedule_products<X::kParts * X::kProducts>();
      }
      schedule_end();
    }
    g_last = g_now;
    g_now = g_next;
    g_next = g_ahead;
    __syncthreads();  // the LDS blocks are read
  }
  if (w == NW / 2) gate(c_first, g_last);

  if (seg == 0 && has_v) {
    const __amdgpu_buffer_rsrc_t to = buffer(A.S + (int64_t)bh * DK * DV, DK * DV * 4);
#pragma unroll
    for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(Gk[kt][i]), to,
                                              (g4 * DV + v0 + col) * 4, (kt * 16 + i) * DV * 4, 0);
  }
}

template <class T, int DK, int DV>
hipError_t launch_backward(const LinearArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((linear_backward_kernel<T, DK, DV>),
                     dim3((unsigned)((int64_t)a.BH * a.nseg)),
                     dim3(BackwardShape<DK, DV>::kThreads), 0, stream, a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_backward_type(const LinearArgs& a, int d_k, int d_v, hipStream_t s) {
  switch (d_k * 1000 + d_v) {
    case 32032: return launch_backward<T, 32, 32>(a, s);
    case 32064: return launch_backward<T, 32, 64>(a, s);
    case 32128: return launch_backward<T, 32, 128>(a, s);
    case 64032: return launch_backward<T, 64, 32>(a, s);
    case 64064: return launch_backward<T, 64, 64>(a, s);
    case 64128: return launch_backward<T, 64, 128>(a, s);
    case 128032: return launch_backward<T, 128, 32>(a, s);
    case 128064: return launch_backward<T, 128, 64>(a, s);
    default: return launch_backward<T, 128, 128>(a, s);
  }
}

}  // namespace lin
}  // namespace sdm
