// The dense recurrence with a decay for each head, in chunks (forward):
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   out_t = S_t^T q_t.
// With L_t the sum of g over the chunk's steps through t, S the state before
// the chunk and C its last step:
//   out_t = exp(L_t) S^T q_t + sum over s <= t of exp(L_t - L_s) (q_t . k_s) v_s
//   S'    = exp(L_C) S       + sum over s of exp(L_C - L_s) k_s v_s^T
// (all exponents <= 0 for decays), as products of 16 x 16 tiles.
//
// One workgroup of four wavefronts walks the chunks of a memory, or of one
// segment of it; the state stays in its accumulators, each wavefront holding
// all d_k rows of d_v / 4 columns.  Where memories are few, the steps are cut
// into segments: a first kernel (modes 1 and 2) finds what each segment adds to
// the state, another adds these up (linear.hip), then each segment starts from
// its own state.
#pragma once
#include "dense.h"
#include "linear_tile.h"

namespace sdm {
namespace lin {

constexpr int kScanThreads = 256;

template <class T, int DK, int DV, int MODE>
__global__ __launch_bounds__(kScanThreads) void linear_kernel(LinearArgs A) {
  typedef Tile<T> X;
  typedef typename X::Frag Frag;
  constexpr int C = X::kChunk;
  constexpr bool kOut = MODE == 0;   // outputs, not the state alone
  constexpr bool kReverse = MODE == 2;
  typedef Block<T, DK, kScanThreads> BlockK;
  typedef Block<T, DV, kScanThreads> BlockV;
  constexpr int ldk = BlockK::kLd, ldv = BlockV::kLd, ldp = C + X::kPad;
  constexpr int kTT = C / 16;                       // tiles of steps
  constexpr int kKT = DK / 16;                      // tiles of state rows
  constexpr int kCT = DV >= 64 ? DV / 64 : 1;       // tiles of state columns per wavefront
  __shared__ __align__(16) T sq[kOut ? C * ldk : 8];
  __shared__ __align__(16) T sk[C * ldk];
  __shared__ __align__(16) T sv[C * ldv];
  __shared__ __align__(16) T sp[kOut ? C * ldp : 8];  // q_t . k_s and its decay, rows t
  __shared__ Decays<C> sd[2];

  const int lane = lane_id(), col = lane & 15, g4 = 4 * (lane >> 4);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t pid = xcd_contiguous(blockIdx.x, gridDim.x);
  const int bh = (int)(pid / A.nseg), seg = (int)(pid % A.nseg);
  const int c_first = seg * A.seg_chunks;
  const int c_end = c_first + A.seg_chunks < A.nchunk ? c_first + A.seg_chunks : A.nchunk;
  const int n = c_end - c_first;
  if (!kOut && (kReverse ? seg == 0 : seg == A.nseg - 1)) return;  // no segment follows it
  const int64_t key_row = (int64_t)(bh / A.share) * A.T, row = (int64_t)bh * A.T;
  const T* gq = kOut ? (const T*)A.q + key_row * DK : nullptr;
  const T* gk = (kReverse ? (const T*)A.q : (const T*)A.k) + key_row * DK;
  const T* gv = (kReverse ? (const T*)A.dout : (const T*)A.v) + row * DV;
  const float* gg = A.g + row;

  const int ct0 = w * kCT;  // first of this wavefront's column tiles
  const bool mine = ct0 < DV / 16;
  f32x4 S[kKT][kCT];
  const float* from = nullptr;
  if (kOut) from = A.nseg > 1 ? A.seg_state + ((int64_t)bh * A.nseg + seg) * DK * DV
                              : A.S + (int64_t)bh * DK * DV;
#pragma unroll
  for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
    for (int ct = 0; ct < kCT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        S[kt][ct][i] = kOut && mine ? from[(kt * 16 + g4 + i) * DV + (ct0 + ct) * 16 + col] : 0.0f;

  BlockK bq, bk;
  BlockV bv;
  auto chunk_of = [&](int i) { return kReverse ? c_end - 1 - i : c_first + i; };
  auto rows_of = [&](int c) {
    const int64_t left = A.T - (int64_t)c * C;
    return left < C ? (int)left : C;
  };
  auto load = [&](int c) {
    const int64_t t0 = (int64_t)c * C;
    const int valid = rows_of(c);
    if (kOut) bq.load(gq + t0 * DK, valid);
    bk.load(gk + t0 * DK, valid);
    bv.load(gv + t0 * DV, valid);
  };
  auto step_log = [&](int c) {  // of step `lane`
    return lane < rows_of(c) ? log2_decay(gg[(int64_t)c * C + lane]) : 0.0;
  };
  double total = 0.0;
  load(chunk_of(0));
  if (w == 0) total = scan_decays<C>(step_log(chunk_of(0)), sd[0]);

  for (int i = 0; i < n; ++i) {
    const int c = chunk_of(i);
    const Decays<C>& d = sd[i & 1];
    if (kOut) bq.store(sq);
    bk.store(sk);
    bv.store(sv);
    __syncthreads();
    double next_log = 0.0;
    if (i + 1 < n) {
      load(chunk_of(i + 1));
      if (w == 0) next_log = step_log(chunk_of(i + 1));
    }
    if (kOut) {
      // this wavefront's tiles of (q_t . k_s) decay(s, t), s <= t, in rows s:
      // four consecutive s of step t per lane
      constexpr int kUnits = kTT == 4 ? 4 : 1;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int tt = kTT == 4 ? w : w >> 1, st = kTT == 4 ? u : w & 1;
        if (st > (tt | 1)) continue;  // no product below reads it
        f32x4 p = {0, 0, 0, 0};
        if (st <= tt) {
#pragma unroll
          for (int kb = 0; kb < DK / 32; ++kb)
            p = X::mma(X::rows(sk, ldk, st * 16, kb * 32), X::rows(sq, ldk, tt * 16, kb * 32), p);
          const int t = tt * 16 + col, s = st * 16 + g4;
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = s + j <= t ? p[j] * decay_between<C>(d, t, s + j) : 0.0f;
        }
        X::store4(sp + (tt * 16 + col) * ldp + st * 16 + g4, p);
      }
    }
    if (i + 1 < n && w == 0) total += scan_decays<C>(next_log, sd[(i + 1) & 1]);
    if (kOut) __syncthreads();
    if (mine) {
      if (kOut && A.tape) {
        float* tape = A.tape + ((int64_t)bh * A.nchunk + c) * DK * DV;
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int ct = 0; ct < kCT; ++ct)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tape[(kt * 16 + g4 + j) * DV + (ct0 + ct) * 16 + col] = S[kt][ct][j];
      }
      Frag V[kCT][C / 32];
#pragma unroll
      for (int ct = 0; ct < kCT; ++ct)
#pragma unroll
        for (int sb = 0; sb < C / 32; ++sb) V[ct][sb] = X::cols(sv, ldv, sb * 32, (ct0 + ct) * 16);
      if (kOut) {
        // outputs transposed: rows are columns of v, so a lane holds four
        // consecutive values of step t.  The state enters rounded to T (bf16: the
        // outputs are rounded to it as well), the accumulators keep fp32.
        const int64_t t0 = (int64_t)c * C;
        const int valid = rows_of(c);
        f32x4 o[kTT][kCT];
#pragma unroll
        for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
          for (int ct = 0; ct < kCT; ++ct) o[tt][ct] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) {
          Frag s[kCT];
#pragma unroll
          for (int ct = 0; ct < kCT; ++ct) s[ct] = X::pack(S[2 * kb][ct], S[2 * kb + 1][ct]);
#pragma unroll
          for (int tt = 0; tt < kTT; ++tt) {
            const Frag q = X::rows(sq, ldk, tt * 16, kb * 32);
#pragma unroll
            for (int ct = 0; ct < kCT; ++ct) o[tt][ct] = X::mma(s[ct], q, o[tt][ct]);
          }
        }
#pragma unroll
        for (int tt = 0; tt < kTT; ++tt) {
          const float into = d.into[tt * 16 + col];
#pragma unroll
          for (int ct = 0; ct < kCT; ++ct) o[tt][ct] *= into;
#pragma unroll
          for (int sb = 0; sb <= tt / 2; ++sb) {
            const Frag p = X::rows(sp, ldp, tt * 16, sb * 32);
#pragma unroll
            for (int ct = 0; ct < kCT; ++ct) o[tt][ct] = X::mma(V[ct][sb], p, o[tt][ct]);
          }
          const int t = tt * 16 + col;
          if (t < valid) {
            T* out = (T*)A.out + (row + t0 + t) * DV;
#pragma unroll
            for (int ct = 0; ct < kCT; ++ct) X::store4(out + (ct0 + ct) * 16 + g4, o[tt][ct]);
          }
        }
      }
      // the state: v (dout in reverse) scaled by its decay, in parts
      const float* scale = kReverse ? d.into : d.onto;
      Frag part[kCT][C / 32][X::kParts];
#pragma unroll
      for (int sb = 0; sb < C / 32; ++sb) {
        f32x8 a;
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = scale[sb * 32 + 16 * (j / 4) + g4 + j % 4];
#pragma unroll
        for (int ct = 0; ct < kCT; ++ct) X::split(X::widen(V[ct][sb]) * a, part[ct][sb]);
      }
      const float whole = d.whole;
#pragma unroll
      for (int kt = 0; kt < kKT; ++kt) {
#pragma unroll
        for (int ct = 0; ct < kCT; ++ct) S[kt][ct] *= whole;
#pragma unroll
        for (int sb = 0; sb < C / 32; ++sb) {
          const Frag k = X::cols(sk, ldk, sb * 32, kt * 16);
#pragma unroll
          for (int p = 0; p < X::kParts; ++p)
#pragma unroll
            for (int ct = 0; ct < kCT; ++ct) S[kt][ct] = X::mma(k, part[ct][sb][p], S[kt][ct]);
        }
      }
    }
    __syncthreads();  // the LDS blocks are read
  }

  float* to = nullptr;
  if (!kOut) {
    to = A.seg_state + ((int64_t)bh * A.nseg + seg) * DK * DV;
    if (threadIdx.x == 0) A.seg_log[(int64_t)bh * A.nseg + seg] = total;
  } else if (seg == A.nseg - 1) {
    to = A.S + (int64_t)bh * DK * DV;
  }
  if (to && mine) {
#pragma unroll
    for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
      for (int ct = 0; ct < kCT; ++ct)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to[(kt * 16 + g4 + i) * DV + (ct0 + ct) * 16 + col] = S[kt][ct][i];
  }
}

template <class T, int DK, int DV>
hipError_t launch_mode(const LinearArgs& a, int mode, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.BH * a.nseg)), block(kScanThreads);
  if (mode == 0)
    hipLaunchKernelGGL((linear_kernel<T, DK, DV, 0>), grid, block, 0, stream, a);
  else if (mode == 1)
    hipLaunchKernelGGL((linear_kernel<T, DK, DV, 1>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((linear_kernel<T, DK, DV, 2>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_scan_type(const LinearArgs& a, int d_k, int d_v, int mode, hipStream_t s) {
  switch (d_k * 1000 + d_v) {
    case 32032: return launch_mode<T, 32, 32>(a, mode, s);
    case 32064: return launch_mode<T, 32, 64>(a, mode, s);
    case 32128: return launch_mode<T, 32, 128>(a, mode, s);
    case 64032: return launch_mode<T, 64, 32>(a, mode, s);
    case 64064: return launch_mode<T, 64, 64>(a, mode, s);
    case 64128: return launch_mode<T, 64, 128>(a, mode, s);
    case 128032: return launch_mode<T, 128, 32>(a, mode, s);
    case 128064: return launch_mode<T, 128, 64>(a, mode, s);
    default: return launch_mode<T, 128, 128>(a, mode, s);
  }
}

}  // namespace lin
}  // namespace sdm
