// Token projections from 4-bit microscaled operands (mx.h): y = Wt x on the
// values the codes stand for, fp32 accumulation, the outputs of project.hip
// (page "Riepilogo Tecnico: Sparse Delta Memory (SDM)", section "Meccanismo
// Core", item 2).  The matrix cores take the codes and the scales as they
// lie in memory: every product of two e2m1 values is exact, and each block of
// 32 products is scaled by 2^(bx + bw - 254) inside the instruction.
//
// Many tokens: project_mx4_kernel, a 256 x 256 tile of tokens x columns per
// 512-thread workgroup, 2 x 4 wavefronts of 128 x 64, each 4 x 2 blocks of
// v_mfma_scale_f32_32x32x64_f8f6f4.  K is taken 256 at a time (128 bytes of
// codes and two 4-byte scale words per row) through two LDS stages filled by
// direct global-to-LDS loads; the 16-byte segments of a row are swizzled so
// that the fragment reads are free of bank conflicts.  Tiles are numbered so
// that each XCD gets a contiguous range, grouped along M.
//
// Few tokens (a decode step): project_mx4_few, bound by streaming the weights
// once.  See there.
#include <type_traits>

#include "internal.h"
#include "mx.h"
#include "project_store.h"

namespace sdm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kXBM = kProjTile, kXBN = kProjTile;  // output tile
constexpr int kXBK = 256;                           // K per stage
constexpr int kXRow = kXBK / 2;                     // code bytes of a row in a stage
constexpr int kXThreads = 512;                      // 8 wavefronts
constexpr int kXWavesM = 2;                         // wavefront grid 2 (M) x 4 (N)
constexpr int kXTM = 4, kXTN = 2;                   // 32 x 32 blocks per wavefront
constexpr int kXSegs = kXRow / 16;                  // 16-byte segments per row
constexpr int kXCodes = (kXBM + kXBN) * kXRow;      // code bytes per stage
constexpr int kXScales = 2 * (kXBM + kXBN) * 4;     // scale bytes per stage: 2 words per row
constexpr int kXStage = kXCodes + kXScales;
constexpr int kXLoads = kXBM * kXSegs / kXThreads;  // 16-byte loads per thread, operand, stage
constexpr int kXGroupM = 8;
static_assert(kXLoads == 4 && kXSegs == 8, "the slot numbering assumes 4 loads of 8 segments");
static_assert(kXScales == 2 * kXThreads * 4, "two scale words per thread and stage");
static_assert(2 * kXStage <= 160 * 1024, "two stages in LDS");

struct Mx4Args {
  const uint8_t *Xq, *Xs, *Wq, *Ws;
  int K;
  int nbm, nbn;
  ProjOut out;
};

// position of 16-byte segment `seg` in row `row` of a stage
__device__ __forceinline__ int seg_pos(int row, int seg) { return seg ^ ((row >> 1) & 7); }

// s_waitcnt with only the vector-memory count limited: vmcnt(n), n < 16
constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8); }

// a workgroup barrier without a memory fence (the direct loads are waited for
// by count just before it); the empty asm keeps LDS accesses on their side
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// fp4 operands use the first four words of the instruction's eight
__device__ __forceinline__ i32x8 widen(const i32x4& q) {
  return __builtin_shufflevector(q, q, 0, 1, 2, 3, -1, -1, -1, -1);
}

constexpr int kFp4 = 4;  // element format code of the f8f6f4 instructions

template <int SEL>
__device__ __forceinline__ f32x16 mfma32(const i32x4& a, const i32x4& b, const f32x16& c, int sa,
                                         int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, SEL,
                                                         sa, SEL, sb);
}

// A wavefront's fragments of 64 columns, and its scale words of 128.
struct Frags {
  i32x4 a[kXTM], b[kXTN];
};
struct Scales {
  int a[kXTM], b[kXTN];
};

__global__ __launch_bounds__(kXThreads) void project_mx4_kernel(Mx4Args A) {
  __shared__ __align__(16) uint8_t lds[2 * kXStage];
  const int tid = threadIdx.x, lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int64_t M = A.out.M, Ncols = A.out.Ncols;

  const int64_t nblocks = (int64_t)A.nbm * A.nbn;
  int64_t pid = blockIdx.x;
  if (nblocks % 8 == 0) pid = (pid & 7) * (nblocks / 8) + (pid >> 3);  // a contiguous range per XCD
  const int64_t per_group = (int64_t)kXGroupM * A.nbn;
  const int64_t first_m = (pid / per_group) * kXGroupM;
  const int64_t gsz = (A.nbm - first_m) < kXGroupM ? (A.nbm - first_m) : kXGroupM;
  const int64_t pm = first_m + (pid % per_group) % gsz;
  const int64_t pn = (pid % per_group) / gsz;
  const int64_t m0 = pm * kXBM, n0 = pn * kXBN;

  // Direct loads.  Codes: load q of wavefront w fills the 64 consecutive
  // 16-byte slots (q * 8 + w) * 64 + lane; slot s is position s % 8 of row
  // s / 8, whose swizzle is the same for every q.  Scales: thread i < 256
  // (>= 256) loads row i % 256's word of the stage's first (second) 128
  // columns.  Rows past the matrix read its last row (their products land
  // only in outputs that are never stored).  Offsets are from the tile's
  // first row: 32 bits (256 rows of at most 32 KiB).
  const int nk = (A.K + kXBK - 1) / kXBK;
  const bool half = A.K % kXBK != 0;  // the last stage holds 128 columns
  const uint32_t row_bytes = (uint32_t)A.K / 2;
  const int mrows = (int)(M - m0 < kXBM ? M - m0 : kXBM);
  const int nrows = (int)(Ncols - n0 < kXBN ? Ncols - n0 : kXBN);
  const int row0 = w * 8 + lane / kXSegs, seg = seg_pos(row0, lane % kXSegs);
  uint32_t srcA[kXLoads], srcB[kXLoads];
#pragma unroll
  for (int q = 0; q < kXLoads; ++q) {
    const int row = q * 64 + row0;
    srcA[q] = (uint32_t)(row < mrows ? row : mrows - 1) * row_bytes + seg * 16;
    srcB[q] = (uint32_t)(row < nrows ? row : nrows - 1) * row_bytes + seg * 16;
  }
  const uint8_t *tileA = A.Xq + m0 * row_bytes, *tileB = A.Wq + n0 * row_bytes;
  const int srow = tid & 255, g0 = w >> 2;
  const uint32_t sA = (uint32_t)(srow < mrows ? srow : mrows - 1) * 4;
  const uint32_t sB = (uint32_t)(srow < nrows ? srow : nrows - 1) * 4;
  const uint8_t *tileXs = A.Xs + m0 * 4, *tileWs = A.Ws + n0 * 4;
  // Load stage kt into its buffer (past the last stage: the last one again,
  // into a buffer no longer read, so that the loop has no branch).  In a half
  // stage the second half's slots repeat the first (not read).
  auto issue = [&](int kt) __attribute__((always_inline)) {
    uint8_t* base = lds + (kt & 1) * kXStage;
    kt = kt < nk ? kt : nk - 1;
    const bool cut = half && kt == nk - 1;
    const uint32_t back = cut && seg >= kXSegs / 2 ? kXRow / 2 : 0;
    const uint8_t *pa = tileA + (int64_t)kt * kXRow, *pb = tileB + (int64_t)kt * kXRow;
#pragma unroll
    for (int q = 0; q < kXLoads; ++q) {
      __builtin_amdgcn_global_load_lds((const void*)(pa + (srcA[q] - back)),
                                       (void*)(base + (q * 8 + w) * kWave * 16), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const void*)(pb + (srcB[q] - back)),
                                       (void*)(base + kXBM * kXRow + (q * 8 + w) * kWave * 16),
                                       16, 0, 0);
    }
    const int64_t g = 2 * (int64_t)kt + (cut ? 0 : g0);
    __builtin_amdgcn_global_load_lds((const void*)(tileXs + g * M * 4 + sA),
                                     (void*)(base + kXCodes + w * kWave * 4), 4, 0, 0);
    __builtin_amdgcn_global_load_lds((const void*)(tileWs + g * Ncols * 4 + sB),
                                     (void*)(base + kXCodes + (kXThreads + w * kWave) * 4), 4, 0,
                                     0);
  };

  const int wm = w % kXWavesM, wn = w / kXWavesM;  // this wavefront's 128 x 64 part of the tile
  const int lr = lane & 31, lh = lane >> 5;
  // Fragment of 64 columns: lane l holds columns 32 * (l / 32) .. + 31 of row
  // l % 32, i.e. segment 2 * kk + l / 32 of the stage's row; its scale is
  // byte 2 * (kk % 2) + l / 32 of word kk / 2, taken after a shift by l / 32
  // bytes as byte 2 * (kk % 2) of every lane.  The next 32 rows lie 4096
  // bytes on (the swizzle repeats every 16 rows).
  const int rowA = wm * kXTM * 32 + lr, rowB = wn * kXTN * 32 + lr;
  const int offA = rowA * kXRow + seg_pos(rowA, lh) * 16;
  const int offB = kXBM * kXRow + rowB * kXRow + seg_pos(rowB, lh) * 16;
  const int scA = kXCodes + rowA * 4, scB = kXCodes + kXThreads * 4 + rowB * 4;
  f32x16 acc[kXTM][kXTN];
#pragma unroll
  for (int i = 0; i < kXTM; ++i)
#pragma unroll
    for (int j = 0; j < kXTN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Two sets of fragments: while the matrix cores take one, the next 64
  // columns' are read from LDS into the other, across the stage boundary too.
  Frags fr[2];
  Scales sc[2];
  auto read = [&](int kt, int kk) __attribute__((always_inline)) {
    const uint8_t* base = lds + (kt & 1) * kXStage;
    const uint8_t *pa = base + (offA ^ (kk * 32)), *pb = base + (offB ^ (kk * 32));
    Frags& f = fr[kk & 1];
    if (kk % 2 == 0) {
      Scales& s = sc[kk / 2];
#pragma unroll
      for (int j = 0; j < kXTN; ++j)
        s.b[j] = *reinterpret_cast<const int*>(base + scB + (kk / 2) * 1024 + j * 128);
#pragma unroll
      for (int i = 0; i < kXTM; ++i)
        s.a[i] = *reinterpret_cast<const int*>(base + scA + (kk / 2) * 1024 + i * 128);
    }
#pragma unroll
    for (int j = 0; j < kXTN; ++j) f.b[j] = *reinterpret_cast<const i32x4*>(pb + j * 32 * kXRow);
#pragma unroll
    for (int i = 0; i < kXTM; ++i) f.a[i] = *reinterpret_cast<const i32x4*>(pa + i * 32 * kXRow);
  };
  auto mul = [&](int kk) __attribute__((always_inline)) {
    const Frags& f = fr[kk & 1];
    Scales& s = sc[kk / 2];
    if (kk % 2 == 0) {
#pragma unroll
      for (int j = 0; j < kXTN; ++j) s.b[j] >>= 8 * lh;
#pragma unroll
      for (int i = 0; i < kXTM; ++i) s.a[i] >>= 8 * lh;
    }
#pragma unroll
    for (int i = 0; i < kXTM; ++i)
#pragma unroll
      for (int j = 0; j < kXTN; ++j)
        acc[i][j] = kk % 2 == 0 ? mfma32<0>(f.a[i], f.b[j], acc[i][j], s.a[i], s.b[j])
                                : mfma32<2>(f.a[i], f.b[j], acc[i][j], s.a[i], s.b[j]);
  };
  // One phase: the next fragments' reads go out, then the matrix
  // instructions of the present ones.  (Left to itself the compiler gathers
  // the reads of a whole stage in front, which does not fit the registers.)
  auto phase = [&](int kk, int kt_next, int kk_next) __attribute__((always_inline)) {
    read(kt_next, kk_next);
    __builtin_amdgcn_sched_barrier(0);
    mul(kk);
    __builtin_amdgcn_sched_barrier(0);
  };

  issue(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  stage_barrier();
  issue(1);
  read(0, 0);
  for (int kt = 0; kt < nk - 1; ++kt) {
    phase(0, kt, 1);
    phase(1, kt, 2);
    phase(2, kt, 3);
    // stage kt + 1 is in, and stage kt's last fragments are in registers, for
    // this wavefront; after the barrier for all of them
    __builtin_amdgcn_s_waitcnt(0);
    stage_barrier();
    issue(kt + 2);
    phase(3, kt + 1, 0);
  }
  if (!half) {
    phase(0, nk - 1, 1);
    phase(1, nk - 1, 2);
    phase(2, nk - 1, 3);
    mul(3);
  } else {
    phase(0, nk - 1, 1);
    mul(1);
  }

  // no load may reach LDS after the workgroup has left it
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));

  // lane l, accumulator r of block (i, j) holds C[row][col] with
  // row = 8*(r/4) + 4*(l/32) + r%4 and col = l%32 within the 32 x 32 block
  ProjColumn c[kXTN];
#pragma unroll
  for (int j = 0; j < kXTN; ++j)
    c[j] = project_column(A.out, (uint32_t)(n0 + (wn * kXTN + j) * 32 + lr));
#pragma unroll
  for (int i = 0; i < kXTM; ++i)
    project_store_blocks(A.out, c, m0 + (wm * kXTM + i) * 32, acc[i]);
}

// Few tokens: at most 16 * MT of them against every column.  The weights are
// read once, straight into registers (no LDS: each code is used by one
// wavefront only); the tokens' codes come from L2.  A workgroup owns 16 * CT
// columns and its kFewWaves wavefronts split K in turns of 128 columns, so
// together they walk each weight row in runs of kFewWaves * 64 bytes; each
// keeps kFewAhead turns of loads in flight.  v_mfma_scale_f32_16x16x128_f8f6f4:
// lane l holds columns 32 * (l / 16) .. + 31 of the 128 of row l % 16.  The
// wavefronts' sums meet in LDS and are added in wavefront order (the same
// result every time).
constexpr int kFewWaves = 8;
constexpr int kFewAhead = 4;

template <int MT, int CT>
__global__ __launch_bounds__(kFewWaves* kWave) void project_mx4_few(Mx4Args A) {
  constexpr int kBlocks = MT * CT;                     // 16 x 16 output blocks
  constexpr int kTurn = kBlocks < 4 ? kBlocks : 4;     // of them summed at a time
  __shared__ f32x4 part[kTurn][kFewWaves][kWave];
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lr = lane & 15, lh = lane >> 4;
  const int64_t M = A.out.M, Ncols = A.out.Ncols;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * CT);
  const uint8_t *xq[MT], *xs[MT], *wq[CT], *ws[CT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {  // rows past the end repeat the last one (not stored)
    const int64_t r = 16 * i + lr < M ? 16 * i + lr : M - 1;
    xq[i] = A.Xq + r * (A.K / 2) + lh * 16;
    xs[i] = A.Xs + r * 4 + lh;
  }
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int64_t c = n0 + 16 * j + lr < Ncols ? n0 + 16 * j + lr : Ncols - 1;
    wq[j] = A.Wq + c * (A.K / 2) + lh * 16;
    ws[j] = A.Ws + c * 4 + lh;
  }
  f32x4 acc[MT][CT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int G = A.K / 128;
  auto turns = [&](int g, auto count) __attribute__((always_inline)) {
    constexpr int U = decltype(count)::value;
    i32x4 a[U][MT], b[U][CT];
    int sa[U][MT], sb[U][CT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t gu = g + u * kFewWaves;
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        b[u][j] = *reinterpret_cast<const i32x4*>(wq[j] + gu * 64);
        sb[u][j] = ws[j][gu * Ncols * 4];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        a[u][i] = *reinterpret_cast<const i32x4*>(xq[i] + gu * 64);
        sa[u][i] = xs[i][gu * M * 4];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              widen(a[u][i]), widen(b[u][j]), acc[i][j], kFp4, kFp4, 0, sa[u][i], 0, sb[u][j]);
  };
  int g = w;
  for (; g + (kFewAhead - 1) * kFewWaves < G; g += kFewAhead * kFewWaves)
    turns(g, std::integral_constant<int, kFewAhead>{});
  for (; g < G; g += kFewWaves) turns(g, std::integral_constant<int, 1>{});

  // lane l, value r of block (i, j): token 16 i + 4 (l / 16) + r, column 16 j + l % 16
#pragma unroll
  for (int t = 0; t < kBlocks; t += kTurn) {
    if (t > 0) __syncthreads();
#pragma unroll
    for (int q = 0; q < kTurn; ++q) part[q][w][lane] = acc[(t + q) / CT][(t + q) % CT];
    __syncthreads();
    for (int e = threadIdx.x; e < kTurn * 256; e += kFewWaves * kWave) {
      // element e: block q, value r of lane l; consecutive threads take consecutive columns
      const int q = e / 256, l = (e & 15) | ((e >> 2) & 48), r = (e >> 4) & 3;
      const int i = (t + q) / CT, j = (t + q) % CT;
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < kFewWaves; ++k) y += part[q][k][l][r];
      const int64_t row = 16 * i + 4 * (l >> 4) + r, col = n0 + 16 * j + (l & 15);
      if (row < M && col < Ncols) project_store_one(A.out, project_column(A.out, (uint32_t)col),
                                                     project_token(A.out, (uint32_t)row), y);
    }
  }
}

template <int MT, int CT>
void launch_few(const Mx4Args& A, hipStream_t stream) {
  const int64_t blocks = (A.out.Ncols + 16 * CT - 1) / (16 * CT);
  hipLaunchKernelGGL((project_mx4_few<MT, CT>), dim3((unsigned)blocks), dim3(kFewWaves * kWave), 0,
                     stream, A);
}

}  // namespace

hipError_t launch_project_mx4(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                              const uint8_t* Ws, int B, int T, int d_model, int H, int n, int d_v,
                              float* s1, float* s2, float* q1, float* q2, float* v, float* alpha,
                              float* beta, hipStream_t stream) {
  Mx4Args A;
  A.Xq = Xq;
  A.Xs = Xs;
  A.Wq = Wq;
  A.Ws = Ws;
  A.K = d_model;
  A.out = project_out(B, T, H, n, d_v, s1, s2, q1, q2, v, alpha, beta);
  if (A.out.M == 0) return hipSuccess;
  if (A.out.M <= kProjFewTokens) {
    const int mt = (int)((A.out.M + 15) / 16);
    if (mt == 1)
      launch_few<1, 1>(A, stream);
    else if (mt == 2)
      launch_few<2, 2>(A, stream);
    else
      launch_few<4, 4>(A, stream);
    return hipGetLastError();
  }
  A.nbm = (int)((A.out.M + kXBM - 1) / kXBM);
  A.nbn = (int)((A.out.Ncols + kXBN - 1) / kXBN);
  const int64_t blocks = project_blocks(A.out.M, A.out.Ncols);
  hipLaunchKernelGGL(project_mx4_kernel, dim3((unsigned)blocks), dim3(kXThreads), 0, stream, A);
  return hipGetLastError();
}

}  // namespace sdm
