// The dense recurrence with a decay for each head, in chunks (forward):
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   out_t = S_t^T q_t.
// With L_t the sum of g over the chunk's steps through t, S the state before
// the chunk and C its last step:
//   out_t = exp(L_t) S^T q_t + sum over s <= t of exp(L_t - L_s) (q_t . k_s) v_s
//   S'    = exp(L_C) S       + sum over s of exp(L_C - L_s) k_s v_s^T
// (all exponents <= 0 for decays), as products of 16 x 16 tiles.
//
// One workgroup walks the chunks of a memory, or of one segment of it; the
// state stays in its accumulators, each of four wavefronts holding all d_k rows
// of a quarter of the columns (at least 16).  Where memories are few, the steps are cut
// into segments: a first kernel (modes 1 and 2) finds what each segment adds to
// the state, another adds these up (linear.hip), then each segment starts from
// its own state.
//
// Bound by the phases of a chunk, which follow each other (LDS stores, q.k,
// outputs, state): 128 x 128 bf16, 64 memories x 4096 steps in four segments,
// 33 us for the segments' states and 92 for the scan (6 us a chunk of 64 steps),
// where its bytes need 40; 512 memories x 2048 steps 300 us (3.8 TB/s), since two
// workgroups a compute unit then fill each other's waits, held back by power
// (1.45 GHz) and LDS.  fp32, 64 x 128, 32 memories x 2047 steps in eight segments:
// 17 + 40 us; a chunk of 32 steps there is eight times the matrix instructions of
// bf16's, at twice the cycles each.  bf16's second parts of the state and of the
// pairs, without which outputs are 1.4 times as far from the exact ones, cost 12 of
// the 92 us.  Four wavefronts of 32 columns read each fragment of q and k for two
// products: eight wavefronts of 16 read LDS twice as often (with one part each, 64 x
// 4096 141 us; 117).  One set of LDS blocks, the next chunk's loads in registers:
// two sets need one barrier less but leave room for one workgroup a compute unit
// (with one part each 125 us).
#pragma once
#include "dense.h"
#include "linear_tile.h"

namespace sdm {
namespace lin {

constexpr int kScanWaves = 4, kScanThreads = kScanWaves * kWave;

// MODE: 0 the scan, 3 the scan that keeps its tape, 1 and 2 the state alone,
// forward and in reverse.
template <class T, int DK, int DV, int MODE>
__global__ __launch_bounds__(kScanThreads, 2) void linear_kernel(LinearArgs A) {
  typedef Tile<T> X;
  typedef typename X::Frag Frag;
  constexpr int C = X::kChunk;
  constexpr bool kOut = MODE == 0 || MODE == 3;  // outputs, not the state alone
  constexpr bool kTape = MODE == 3;
  constexpr bool kReverse = MODE == 2;
  constexpr int NW = kScanWaves, NT = kScanThreads;
  typedef Block<T, DK, NT> BlockK;
  typedef Block<T, DV, NT> BlockV;
  typedef Pairs<T> P;
  constexpr int kTT = C / 16;                       // tiles of steps
  constexpr int kKT = DK / 16;                      // tiles of state rows
  constexpr int kCT = DV > 16 * NW ? DV / (16 * NW) : 1;  // tiles of state columns per wavefront
  __shared__ __align__(16) T sq[kOut ? BlockK::kSize : 8];
  __shared__ __align__(16) T sk[BlockK::kSize];
  __shared__ __align__(16) T sv[BlockV::kSize];
  __shared__ __align__(16) T sp[kOut ? P::kParts * P::kSize : 8];  // (q_t . k_s) decay(s, t)
  __shared__ Decays<C> sd[2];
  __shared__ float sg[C];  // g of the next chunk

  const int lane = lane_id(), col = lane & 15, g4 = 4 * (lane >> 4);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t pid = xcd_contiguous(blockIdx.x, gridDim.x);
  const int bh = (int)(pid / (uint32_t)A.nseg), seg = (int)(pid % (uint32_t)A.nseg);
  const int c_first = seg * A.seg_chunks;
  const int c_end = c_first + A.seg_chunks < A.nchunk ? c_first + A.seg_chunks : A.nchunk;
  const int n = c_end - c_first;
  if (!kOut && (kReverse ? seg == 0 : seg == A.nseg - 1)) {
    // no segment follows it: the call's state takes its place, since the scan
    // overwrites that while other segments may not have read it
    const f32x4* own = reinterpret_cast<const f32x4*>(A.S + (int64_t)bh * DK * DV);
    f32x4* copy = reinterpret_cast<f32x4*>(A.seg_state + ((int64_t)bh * A.nseg + seg) * DK * DV);
    for (int i = threadIdx.x; i < DK * DV / 4; i += NT) copy[i] = own[i];
    return;
  }
  const int64_t key_row = (int64_t)(bh / A.share) * A.T, row = (int64_t)bh * A.T;
  const T* gq = kOut ? (const T*)A.q + key_row * DK : nullptr;
  const T* gk = (kReverse ? (const T*)A.q : (const T*)A.k) + key_row * DK;
  const T* gv = (kReverse ? (const T*)A.dout : (const T*)A.v) + row * DV;
  const float* gg = A.g + row;

  const int v0 = w * kCT * 16;  // this wavefront holds columns v0 .. v0 + 16 kCT - 1
  const bool mine = v0 < DV;
  f32x4 S[kKT][kCT];
  auto add_state = [&](const float* from, float decay) {  // S = decay S + from
    const __amdgpu_buffer_rsrc_t b = buffer(from, DK * DV * 4);
#pragma unroll
    for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
      for (int ct = 0; ct < kCT; ++ct)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          S[kt][ct][i] = S[kt][ct][i] * decay + buffer_float(b, (g4 * DV + v0 + col) * 4 + ct * 64,
                                                             (kt * 16 + i) * DV * 4);
  };
#pragma unroll
  for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
    for (int ct = 0; ct < kCT; ++ct) S[kt][ct] = f32x4{0, 0, 0, 0};
  auto store_rows = [&](__amdgpu_buffer_rsrc_t to, int kt) {
#pragma unroll
    for (int ct = 0; ct < kCT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[kt][ct][i]), to,
                                              (g4 * DV + v0 + col) * 4 + ct * 64,
                                              (kt * 16 + i) * DV * 4, 0);
  };

  BlockK bq, bk;
  BlockV bv;
  // The state alone is one weighted sum over the segment's steps, by decays to its
  // end (from its start, in reverse); chunks are taken from there.
  constexpr bool kBack = MODE == 1;
  auto chunk_of = [&](int i) { return kBack ? c_end - 1 - i : c_first + i; };
  // steps of the i-th chunk, 0 behind the last one
  auto rows_of = [&](int i) {
    const int64_t left = A.T - (int64_t)chunk_of(i) * C;
    return i >= n ? 0 : left < C ? (int)left : C;
  };
  auto load = [&](int i) {
    const int64_t t0 = (int64_t)chunk_of(i) * C;
    const int valid = rows_of(i);
    if (kOut) bq.load(gq + t0 * DK, valid);
    bk.load(gk + t0 * DK, valid);
    bv.load(gv + t0 * DV, valid);
  };
  auto g_of = [&](int i) {  // of step `lane` of the i-th chunk
    return __builtin_bit_cast(
        float, __builtin_amdgcn_raw_buffer_load_b32(
                   buffer(gg + (int64_t)chunk_of(i) * C, (uint32_t)rows_of(i) * 4), lane * 4, 0, 0));
  };
  double total = 0.0;
  load(0);
  if (kOut && mine) {
    const float* states = A.seg_state + (int64_t)bh * A.nseg * DK * DV;
    if (A.nseg == 1) {
      add_state(A.S + (int64_t)bh * DK * DV, 0.0f);
    } else if (A.nseg > kOwnSegments) {
      add_state(states + (int64_t)seg * DK * DV, 0.0f);
    } else {
      add_state(states + (int64_t)(A.nseg - 1) * DK * DV, 0.0f);  // the call's state
      for (int i = 0; i < seg; ++i)
        add_state(states + (int64_t)i * DK * DV, pow2((float)A.seg_log[(int64_t)bh * A.nseg + i]));
    }
  }
  if (w == NW - 1) total = scan_decays<C>(log2_decay(g_of(0)), sd[0]);
  float step_g = g_of(1);
#pragma unroll
  for (int kt = 0; kt < kKT; ++kt) arrive(S[kt]);

  for (int i = 0; i < n; ++i) {
    const int c = chunk_of(i);
    const Decays<C>& d = sd[i & 1];
    if (kOut) bq.store(sq);
    bk.store(sk);
    bv.store(sv);
    if (w == NW - 1 && lane < C) sg[lane] = step_g;
    __syncthreads();
    load(i + 1);
    step_g = g_of(i + 2);
    if (kOut) {
      // (q_t . k_s) decay(s, t), s <= t: this wavefront's tiles in rows s, four
      // consecutive s of step t per lane
      constexpr int kUnits = kTT == 4 ? 12 : 4;  // tiles that a product below reads
      static_assert(kUnits % NW == 0, "as many for every wavefront");
#pragma unroll
      for (int u0 = 0; u0 < kUnits; u0 += NW) {
        const int u = u0 + w;
        const int tt = u < 4 ? u >> 1 : 2 + ((u - 4) >> 2), st = u < 4 ? u & 1 : (u - 4) & 3;
        f32x4 p = {0, 0, 0, 0};
        const int t = tt * 16 + col, s = st * 16 + g4;
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb)
          p = X::mma(X::template rows<DK>(sk, st * 16, kb * 32),
                     X::template rows<DK>(sq, tt * 16, kb * 32), p);
        p = decayed(p, decay_between<C>(d, t, s), t, s);
        P::store4(sp, t, s, p);
      }
      __syncthreads();
    }
    if (w == NW - 1)
      total += scan_decays<C>(lane < C ? log2_decay(sg[lane]) : 0.0, sd[(i + 1) & 1],
                              kOut ? 0.0 : total, kOut ? 0.0 : total);
    if (mine) {
      Frag V[kCT][C / 32];
      schedule_end();
      if (kOut) {
        // outputs transposed: rows are columns of v, so a lane holds four
        // consecutive values of step t.  The state enters in kOutParts operands, the
        // accumulators keep fp32.
        const __amdgpu_buffer_rsrc_t out = buffer((T*)A.out + (row + (int64_t)c * C) * DV,
                                                  (uint32_t)(rows_of(i) * DV * (int)sizeof(T)));
        f32x4 o[kTT][kCT];
#pragma unroll
        for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
          for (int ct = 0; ct < kCT; ++ct) o[tt][ct] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) {
          Frag q[kTT];
#pragma unroll
          for (int tt = 0; tt < kTT; ++tt) q[tt] = X::template rows<DK>(sq, tt * 16, kb * 32);
#pragma unroll
          for (int ct = 0; ct < kCT; ++ct) {
            Frag s[X::kOutParts];
            X::template split<X::kOutParts>(Tile<float>::pack(S[2 * kb][ct], S[2 * kb + 1][ct]), s);
#pragma unroll
            for (int j = 0; j < X::kOutParts; ++j)
#pragma unroll
              for (int tt = 0; tt < kTT; ++tt) o[tt][ct] = X::mma(s[j], q[tt], o[tt][ct]);
          }
        }
        // reads one block of products ahead
        schedule_reads<kTT * X::kRowReads>();
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) {
          schedule_reads<kTT * X::kRowReads>();
          schedule_products<kTT * kCT * X::kOutParts * X::kProducts>();
        }
        schedule_end();
#pragma unroll
        for (int ct = 0; ct < kCT; ++ct)
#pragma unroll
          for (int sb = 0; sb < C / 32; ++sb)
            V[ct][sb] = X::template cols<DV>(sv, sb * 32, v0 + ct * 16);
#pragma unroll
        for (int tt = 0; tt < kTT; ++tt) {
          const float into = d.into[tt * 16 + col];
#pragma unroll
          for (int ct = 0; ct < kCT; ++ct) o[tt][ct] *= into;
#pragma unroll
          for (int sb = 0; sb <= tt / 2; ++sb) {
#pragma unroll
            for (int j = 0; j < P::kParts; ++j) {
              const Frag p = P::rows(sp, j, tt * 16, sb * 32);
#pragma unroll
              for (int ct = 0; ct < kCT; ++ct) o[tt][ct] = X::mma(V[ct][sb], p, o[tt][ct]);
            }
          }
#pragma unroll
          for (int ct = 0; ct < kCT; ++ct)
            X::store4(out, (tt * 16 + col) * DV + v0 + ct * 16 + g4, o[tt][ct]);
        }
      } else {
#pragma unroll
        for (int ct = 0; ct < kCT; ++ct)
#pragma unroll
          for (int sb = 0; sb < C / 32; ++sb)
            V[ct][sb] = X::template cols<DV>(sv, sb * 32, v0 + ct * 16);
      }
      // the state: v (dout in reverse) scaled by its decay, in parts (k is bf16
      // already: the products then hold fp32's precision)
      const float* scale = kReverse ? d.into : d.onto;
      Frag part[kCT][C / 32][X::kParts];
#pragma unroll
      for (int sb = 0; sb < C / 32; ++sb) {
        const f32x8 a = Tile<float>::pack(*reinterpret_cast<const f32x4*>(scale + sb * 32 + g4),
                                          *reinterpret_cast<const f32x4*>(scale + sb * 32 + 16 + g4));
#pragma unroll
        for (int ct = 0; ct < kCT; ++ct) X::split(X::widen(V[ct][sb]) * a, part[ct][sb]);
      }
      const float whole = d.whole;
      // the tape: rows of the state go out between the products, just before they
      // change (64 memories x 2048 steps 57 us, 60 all at once in front of them)
      const __amdgpu_buffer_rsrc_t tape =
          buffer(kTape ? A.tape + ((int64_t)bh * A.nchunk + c) * DK * DV : nullptr,
                 kTape ? DK * DV * 4 : 0);
      schedule_end();
#pragma unroll
      for (int kt = 0; kt < kKT; ++kt) {
        if (kTape) store_rows(tape, kt);
#pragma unroll
        for (int ct = 0; ct < kCT; ++ct)
          if (kOut) S[kt][ct] *= whole;
#pragma unroll
        for (int sb = 0; sb < C / 32; ++sb) {
          const Frag k = X::template cols<DK>(sk, sb * 32, kt * 16);
#pragma unroll
          for (int j = 0; j < X::kParts; ++j)
#pragma unroll
            for (int ct = 0; ct < kCT; ++ct) S[kt][ct] = X::mma(k, part[ct][sb][j], S[kt][ct]);
        }
      }
      if (kTape) schedule_writes<kCT * 4>();
      schedule_reads<2 * X::kColReads>();  // two fragments ahead
#pragma unroll
      for (int i = 0; i < kKT * (C / 32); ++i) {
        schedule_reads<X::kColReads>();
        schedule_products<X::kParts * kCT * X::kProducts>();
        if (kTape) schedule_writes<kCT * 4 / (C / 32)>();
      }
      schedule_end();
    }
    __syncthreads();  // the LDS blocks are read
  }

  float* to = nullptr;
  if (!kOut) {
    to = A.seg_state + ((int64_t)bh * A.nseg + seg) * DK * DV;
    if (threadIdx.x == NT - 1) A.seg_log[(int64_t)bh * A.nseg + seg] = total;
  } else if (seg == A.nseg - 1) {
    to = A.S + (int64_t)bh * DK * DV;
  }
  if (to && mine) {
    const __amdgpu_buffer_rsrc_t state = buffer(to, DK * DV * 4);
#pragma unroll
    for (int kt = 0; kt < kKT; ++kt) store_rows(state, kt);
  }
}

template <class T, int DK, int DV>
hipError_t launch_mode(const LinearArgs& a, int mode, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.BH * a.nseg)), block(kScanThreads);
  if (mode == 0 && a.tape)
    hipLaunchKernelGGL((linear_kernel<T, DK, DV, 3>), grid, block, 0, stream, a);
  else if (mode == 0)
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
