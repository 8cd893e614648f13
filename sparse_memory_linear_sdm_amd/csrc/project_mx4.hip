// Token projections from 4-bit microscaled operands (mx.h): y = Wt x on the
// values the codes stand for, fp32 accumulation, the outputs of project.hip
// (page "Riepilogo Tecnico: Sparse Delta Memory (SDM)", section "Meccanismo
// Core", item 2).  The matrix cores take the codes and the scales as they
// lie in memory: every product of two e2m1 values is exact, and each block of
// 32 products is scaled by 2^(bx + bw - 254) inside the instruction.
//
// Many tokens: project_mx4_kernel, a 256 x 256 tile of tokens x columns per
// 512-thread workgroup, 2 x 4 wavefronts of 128 x 64, each 4 x 2 blocks of
// v_mfma_scale_f32_32x32x64_f8f6f4; or 128 x 128 per 256 threads, 2 x 2
// wavefronts of 64 x 64, where there are too few of the larger (pick_kernel).
// K is taken 128 at a time (64 bytes of codes and a 4-byte scale word per row)
// through a ring of four LDS stages filled by direct global-to-LDS loads, three
// of them in flight; the 16-byte segments of a row are swizzled so that the
// fragment reads are free of bank conflicts.  Tiles are numbered so that each
// XCD gets a contiguous range, grouped 8 deep along M.  Per compute unit and 128
// of K the matrix cores need 1024 cycles, LDS about as many (the reads of eight
// wavefronts and the 34 KB that arrive), so the order inside a stage decides: a
// matrix instruction, then two fragment reads or a load, and so on, against all
// reads first, is 8.1 against 9.3 ms without the outputs.  32768 tokens x 33808
// columns at d_model 16384: 9.1-9.8 ms, 3.7-4.0 PFLOP/s (bf16 tiles: 32 ms).
// What bounds it: with no loads in flight the same loop reaches 5.9, bare
// matrix instructions on random codes 6.3 (8.8 on zeros: the card's power limit
// sets the clock), and the outputs' 4.4 GB take 1.0 ms that nothing overlaps.
//
// Few tokens (a decode step): project_mx4_few, bound by streaming the weights
// once.  See there.
#include "internal.h"
#include "mx.h"
#include "project_store.h"

namespace sdm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kXBK = 128;                           // K per stage
constexpr int kXStages = 4;
constexpr int kXRow = kXBK / 2;                     // code bytes of a row in a stage
constexpr int kXSegs = kXRow / 16;                  // 16-byte segments per row
constexpr int kXGroupM = 8;

// A tile: WM x WN wavefronts of TM x TN blocks of 32 x 32.
template <int WM_, int WN_, int TM_, int TN_>
struct XTile {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  static constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  static constexpr int kCodes = (BM + BN) * kXRow;       // code bytes per stage
  static constexpr int kStage = kCodes + (BM + BN) * 4;  // and a scale word per row
  static constexpr int kLoads = BM * kXSegs / kThreads;  // 16-byte loads per thread, operand, stage
  static constexpr int kIssued = 2 * kLoads + 1;         // loads per wavefront and stage
  static_assert(BM == BN && kLoads == 2 && kXSegs == 4, "the slot numbering");
  static_assert((BM + BN) == kThreads, "a scale word per thread and stage");
  static_assert(kXStages * kStage <= 160 * 1024, "the stages in LDS");
};
using Tile256 = XTile<2, 4, 4, 2>;
using Tile128 = XTile<2, 2, 2, 2>;

// Scheduling of one half stage: a matrix instruction, then one LDS read and
// one memory load while it runs.
template <class X>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < X::TM * X::TN; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS read
    __builtin_amdgcn_sched_group_barrier(0x020, X::TM * X::TN >= 8 ? 1 : 2, 0);  // memory load
  }
  __builtin_amdgcn_sched_barrier(0);
}

struct Mx4Args {
  const uint8_t *Xq, *Xs, *Wq, *Ws;
  int K;
  int nbm, nbn;
  ProjOut out;
};

// position of 16-byte segment `seg` in row `row` of a stage
__device__ __forceinline__ int seg_pos(int row, int seg) { return seg ^ ((row >> 2) & 3); }

// s_waitcnt with only the vector-memory count limited: vmcnt(n), n < 16
constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8); }
// the same, and every LDS access done
constexpr int waitcnt_vm_lgkm0(int n) { return (n & 15) | (7 << 4); }

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
template <class X>
struct Frags {
  i32x4 a[X::TM], b[X::TN];
};
template <class X>
struct Scales {
  int a[X::TM], b[X::TN];
};

template <class X>
__global__ __launch_bounds__(X::kThreads) void project_mx4_kernel(Mx4Args A) {
  constexpr int BM = X::BM, BN = X::BN, TM = X::TM, TN = X::TN, kWaves = X::kWaves;
  __shared__ __align__(16) uint8_t lds[kXStages * X::kStage];
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
  const int64_t m0 = pm * BM, n0 = pn * BN;

  // Direct loads.  Codes: load q of wavefront w fills the 64 consecutive
  // 16-byte slots (q * kWaves + w) * 64 + lane; slot s is position s % 4 of row
  // s / 4, whose swizzle is the same for every q.  Scales: thread i < BM
  // (>= BM) loads token (column) i % BM's word.  Rows past the matrix read
  // its last row (their products land only in outputs that are never stored).
  // Offsets are from the tile's first row: 32 bits (256 rows of at most 32 KiB).
  const int nk = A.K / kXBK;
  const uint32_t row_bytes = (uint32_t)A.K / 2;
  const int mrows = (int)(M - m0 < BM ? M - m0 : BM);
  const int nrows = (int)(Ncols - n0 < BN ? Ncols - n0 : BN);
  const int lrow = w * 16 + lane / kXSegs, seg = seg_pos(lrow, lane % kXSegs);
  uint32_t srcA[X::kLoads], srcB[X::kLoads];
#pragma unroll
  for (int q = 0; q < X::kLoads; ++q) {
    const int row = q * 16 * kWaves + lrow;
    srcA[q] = (uint32_t)(row < mrows ? row : mrows - 1) * row_bytes + seg * 16;
    srcB[q] = (uint32_t)(row < nrows ? row : nrows - 1) * row_bytes + seg * 16;
  }
  const uint8_t *tileA = A.Xq + m0 * row_bytes, *tileB = A.Wq + n0 * row_bytes;
  const int srow = tid & (BM - 1), slim = w < kWaves / 2 ? mrows : nrows;
  const uint32_t srcS = (uint32_t)(srow < slim ? srow : slim - 1) * 4;
  const uint8_t* const tileS = w < kWaves / 2 ? A.Xs + m0 * 4 : A.Ws + n0 * 4;
  const int64_t stepS = (w < kWaves / 2 ? M : Ncols) * 4;
  // Load stage kt into its buffer (past the last stage: the last one again,
  // into a buffer no longer read, so that the loop has no branch).
  auto issue = [&](int kt) __attribute__((always_inline)) {
    uint8_t* base = lds + (kt % kXStages) * X::kStage;
    kt = kt < nk ? kt : nk - 1;
    const uint8_t *pa = tileA + (int64_t)kt * kXRow, *pb = tileB + (int64_t)kt * kXRow;
#pragma unroll
    for (int q = 0; q < X::kLoads; ++q) {
      __builtin_amdgcn_global_load_lds((const void*)(pa + srcA[q]),
                                       (void*)(base + (q * kWaves + w) * kWave * 16), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const void*)(pb + srcB[q]),
                                       (void*)(base + BM * kXRow + (q * kWaves + w) * kWave * 16),
                                       16, 0, 0);
    }
    __builtin_amdgcn_global_load_lds((const void*)(tileS + kt * stepS + srcS),
                                     (void*)(base + X::kCodes + w * kWave * 4), 4, 0, 0);
  };

  const int wm = w % X::WM, wn = w / X::WM;  // this wavefront's 128 x 64 part of the tile
  const int lr = lane & 31, lh = lane >> 5;
  // Fragment of 64 columns: lane l holds columns 32 * (l / 32) .. + 31 of row
  // l % 32, i.e. segment 2 * kk + l / 32 of the stage's row; its scale is
  // byte 2 * kk + l / 32 of the row's word, taken after a shift by l / 32
  // bytes as byte 2 * kk of every lane.  The next 32 rows lie 2048 bytes on
  // (the swizzle repeats every 16 rows).
  const int rowA = wm * TM * 32 + lr, rowB = wn * TN * 32 + lr;
  const int offA = rowA * kXRow + seg_pos(rowA, lh) * 16;
  const int offB = BM * kXRow + rowB * kXRow + seg_pos(rowB, lh) * 16;
  const int scA = X::kCodes + rowA * 4, scB = X::kCodes + BM * 4 + rowB * 4;
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Two sets of fragments and scales: while the matrix cores take one, the
  // next 64 columns' are read from LDS into the other, across the stage
  // boundary too.
  Frags<X> fr[2];
  Scales<X> sc[2];
  auto read = [&](int kt, int kk, int set) __attribute__((always_inline)) {
    const uint8_t* base = lds + (kt % kXStages) * X::kStage;
    const uint8_t *pa = base + (offA ^ (kk * 32)), *pb = base + (offB ^ (kk * 32));
    Frags<X>& f = fr[kk];
    if (kk == 0) {
#pragma unroll
      for (int j = 0; j < TN; ++j) sc[set].b[j] = *reinterpret_cast<const int*>(base + scB + j * 128);
#pragma unroll
      for (int i = 0; i < TM; ++i) sc[set].a[i] = *reinterpret_cast<const int*>(base + scA + i * 128);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) f.b[j] = *reinterpret_cast<const i32x4*>(pb + j * 32 * kXRow);
#pragma unroll
    for (int i = 0; i < TM; ++i) f.a[i] = *reinterpret_cast<const i32x4*>(pa + i * 32 * kXRow);
  };
  auto mul = [&](int kk, int set) __attribute__((always_inline)) {
    const Frags<X>& f = fr[kk];
    Scales<X>& s = sc[set];
    if (kk == 0) {
#pragma unroll
      for (int j = 0; j < TN; ++j) s.b[j] >>= 8 * lh;
#pragma unroll
      for (int i = 0; i < TM; ++i) s.a[i] >>= 8 * lh;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = kk == 0 ? mfma32<0>(f.a[i], f.b[j], acc[i][j], s.a[i], s.b[j])
                            : mfma32<2>(f.a[i], f.b[j], acc[i][j], s.a[i], s.b[j]);
  };
  // One stage: the next fragments' reads go out, then the matrix instructions
  // of the present ones, twice.  (Left to itself the compiler gathers the
  // reads in front, which does not fit the registers.)
  auto stage = [&](int kt, int set) __attribute__((always_inline)) {
    issue(kt + kXStages - 1);  // into the buffer of stage kt - 1, read before the last barrier
    read(kt, 1, set);
    mul(0, set);
    interleave<X>();
    // stage kt + 1 is in, and stage kt's last fragments are in registers, for
    // this wavefront; after the barrier for all of them
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((kXStages - 2) * X::kIssued));
    stage_barrier();
    read(kt + 1, 0, set ^ 1);
    mul(1, set);
    interleave<X>();
  };
#pragma unroll
  for (int kt = 0; kt < kXStages - 1; ++kt) issue(kt);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm((kXStages - 2) * X::kIssued));
  stage_barrier();
  read(0, 0, 0);
  int kt = 0;
  for (; kt + 1 < nk; kt += 2) {
    stage(kt, 0);
    stage(kt + 1, 1);
  }
  if (kt < nk) stage(kt, 0);

  // every direct load has landed and every fragment is read, in all wavefronts:
  // LDS is free for the outputs
  __builtin_amdgcn_s_waitcnt(0);
  stage_barrier();

  // Outputs, 64 rows of the wavefront's 64 columns at a time through its own
  // piece of LDS, from where they go row by row: one column a lane.  lane l,
  // accumulator r of block (i, j) holds C[row][col] with row = 8*(r/4) +
  // 4*(l/32) + r%4 and col = l%32 within the 32 x 32 block.  (Stored straight
  // from the accumulators, every row of a wavefront that has a gate among its
  // columns paid for the logistic function: such a tile's outputs took 15 us,
  // so 4; a call of one round lasts as long as them.)
  static_assert(TN * 32 == kWave && TM % 2 == 0 && kWaves * 64 * kWave * 4 <= kXStages * X::kStage,
                "64 x 64 values of each wavefront in LDS");
  float* const mine = reinterpret_cast<float*>(lds) + w * 64 * kWave;
  const ProjColumn c = project_column(A.out, (uint32_t)(n0 + wn * kWave + lane));
#pragma unroll
  for (int i0 = 0; i0 < TM; i0 += 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          mine[(i * 32 + 8 * (r >> 2) + 4 * lh + (r & 3)) * kWave + j * 32 + lr] = acc[i0 + i][j][r];
    wave_sync();
    project_store_rows(A.out, c, m0 + (wm * TM + i0) * 32, mine);
    wave_sync();
  }
}

// Few tokens: 16 * MT tokens (MT = 4: blocks of 64) against 16 * CT columns
// per workgroup, whose wavefronts split K in turns of 128 columns, so that
// together they walk each row in runs of 512 (256) bytes; no barrier until
// their sums meet in LDS, where they are added in wavefront order (the same
// result every time).  v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds columns
// 32 * (l / 16) .. + 31 of the 128 of row l % 16.
//
// Bound by memory (each weight is read once per 64 tokens), and below that by
// the rate of load instructions: a fragment loaded as the matrix cores want
// it has 16 bytes of another row on every lane, 64 requests, and took 145 us
// for 64 tokens at d_model 16384 x 33808 columns.  So four neighbouring lanes
// load 64 bytes of a row, the turn's fragments pass through the wavefront's own
// piece of LDS (16-byte segments swizzled as in the tiles), and the turn after
// it is in flight in registers: 79 us, 3.9 TB/s; one token, the weights' stream
// and little else, 52 us, 5.7 TB/s.
template <int MT, int CT>
constexpr int few_waves() {  // the accumulators of 4 x 7 blocks and up leave room for four
  return MT * CT >= 28 ? 4 : 8;
}

template <int MT, int CT>
__global__ __launch_bounds__((few_waves<MT, CT>() * kWave)) void project_mx4_few(Mx4Args A) {
  constexpr int kWaves = few_waves<MT, CT>();
  constexpr int NF = MT + CT;                       // fragments of a turn
  constexpr int kBlocks = MT * CT;                  // 16 x 16 output blocks
  constexpr int kTurn = kBlocks % 4 == 0 ? 4 : kBlocks % 3 == 0 ? 3 : kBlocks % 2 == 0 ? 2 : 1;
  constexpr int kMine = NF * 1024 + NF * 64;        // a wavefront's LDS: codes, scale words
  constexpr int kSums = kTurn * kWaves * kWave * 16;
  constexpr int kLoadsW = (16 * CT + kWave - 1) / kWave;  // scale-word loads of the columns
  __shared__ __align__(16) uint8_t lds[kWaves * kMine > kSums ? kWaves * kMine : kSums];
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lr = lane & 15, lh = lane >> 4;
  const int64_t M = A.out.M, Ncols = A.out.Ncols;
  // blocks are dealt to the 8 XCDs in turn: the token blocks of a column block
  // follow each other on one of them, so its weights come from that L2
  const int x = blockIdx.x & 7, rest = blockIdx.x >> 3;
  const int64_t m0 = (int64_t)(rest % A.nbm) * (16 * MT);
  const int64_t n0 = ((int64_t)(rest / A.nbm) * 8 + x) * (16 * CT);
  if (n0 >= Ncols) return;  // whole workgroup leaves together

  // Loads: lane l takes segment (l % 4) ^ swizzle of row l / 4 of a fragment's
  // 16; rows past the end repeat the last one (not stored).  Offsets are from
  // the workgroup's first rows: 32 bits (at most 144 rows of 32 KiB).
  const uint32_t row_bytes = (uint32_t)A.K / 2;
  const int row = lane >> 2, seg = seg_pos(row, lane & 3);
  const int mrows = (int)(M - m0 < 16 * MT ? M - m0 : 16 * MT);
  const int nrows = (int)(Ncols - n0 < 16 * CT ? Ncols - n0 : 16 * CT);
  uint32_t src[NF], srcWs[kLoadsW];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = 16 * (f < MT ? f : f - MT) + row, last = (f < MT ? mrows : nrows) - 1;
    src[f] = (uint32_t)(r < last ? r : last) * row_bytes + seg * 16;
  }
  const uint32_t srcXs = (uint32_t)(lane < mrows ? lane : mrows - 1) * 4;
#pragma unroll
  for (int z = 0; z < kLoadsW; ++z) {
    const int c = z * kWave + lane;
    srcWs[z] = (uint32_t)(c < nrows ? c : nrows - 1) * 4;
  }
  const uint8_t *xq = A.Xq + m0 * row_bytes, *wq = A.Wq + n0 * row_bytes;
  const uint8_t *xs = A.Xs + m0 * 4, *ws = A.Ws + n0 * 4;
  uint8_t* const mine = lds + w * kMine;
  uint32_t* const sx = reinterpret_cast<uint32_t*>(mine + NF * 1024);
  uint32_t* const sw = sx + 16 * MT;
  const int frag = lr * 64 + seg_pos(lr, lh) * 16;
  f32x4 acc[MT][CT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int G = A.K / 128;
  i32x4 next[NF];
  uint32_t nextXs, nextWs[kLoadsW];
  auto load = [&](int g) __attribute__((always_inline)) {
    const int64_t gu = g < G ? g : G - 1;  // past the end: again, not used
#pragma unroll
    for (int f = 0; f < NF; ++f)
      next[f] = *reinterpret_cast<const i32x4*>((f < MT ? xq : wq) + gu * 64 + src[f]);
    nextXs = *reinterpret_cast<const uint32_t*>(xs + gu * M * 4 + srcXs);
#pragma unroll
    for (int z = 0; z < kLoadsW; ++z)
      nextWs[z] = *reinterpret_cast<const uint32_t*>(ws + gu * Ncols * 4 + srcWs[z]);
  };
  load(w);
  for (int g = w; g < G; g += kWaves) {
#pragma unroll
    for (int f = 0; f < NF; ++f) *reinterpret_cast<i32x4*>(mine + f * 1024 + lane * 16) = next[f];
    if (lane < 16 * MT) sx[lane] = nextXs;
#pragma unroll
    for (int z = 0; z < kLoadsW; ++z)
      if (z * kWave + lane < 16 * CT) sw[z * kWave + lane] = nextWs[z];
    load(g + kWaves);
    wave_sync();
    i32x4 a[MT];
    int sa[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      a[i] = *reinterpret_cast<const i32x4*>(mine + i * 1024 + frag);
      sa[i] = reinterpret_cast<const uint8_t*>(sx + 16 * i + lr)[lh];
    }
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      const i32x4 b = *reinterpret_cast<const i32x4*>(mine + (MT + j) * 1024 + frag);
      const int sb = reinterpret_cast<const uint8_t*>(sw + 16 * j + lr)[lh];
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            widen(a[i]), widen(b), acc[i][j], kFp4, kFp4, 0, sa[i], 0, sb);
    }
    wave_sync();
  }

  // lane l, value r of block (i, j): token 16 i + 4 (l / 16) + r, column 16 j + l % 16
  f32x4* const part = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int t = 0; t < kBlocks; t += kTurn) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kTurn; ++q)
      part[(q * kWaves + w) * kWave + lane] = acc[(t + q) / CT][(t + q) % CT];
    __syncthreads();
    for (int e = threadIdx.x; e < kTurn * 256; e += kWaves * kWave) {
      // element e: block q, value r of lane l; consecutive threads take consecutive columns
      const int q = e / 256, l = (e & 15) | ((e >> 2) & 48), r = (e >> 4) & 3;
      const int i = (t + q) / CT, j = (t + q) % CT;
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) y += part[(q * kWaves + k) * kWave + l][r];
      const int tok = 16 * i + 4 * (l >> 4) + r, col = 16 * j + (l & 15);
      if (tok < mrows && col < nrows)
        project_store_one(A.out, project_column(A.out, (uint32_t)(n0 + col)),
                          project_token(A.out, (uint32_t)(m0 + tok)), y);
    }
  }
}

template <int MT, int CT>
void launch_few(Mx4Args A, hipStream_t stream) {
  A.nbm = (int)((A.out.M + 16 * MT - 1) / (16 * MT));
  const int64_t cols = (A.out.Ncols + 16 * CT - 1) / (16 * CT);
  hipLaunchKernelGGL((project_mx4_few<MT, CT>), dim3((unsigned)((cols + 7) / 8 * 8 * A.nbm)),
                     dim3(few_waves<MT, CT>() * kWave), 0, stream, A);
}

template <int MT>
void launch_few_columns(const Mx4Args& A, int ct, hipStream_t stream) {
  if (ct == 1) return launch_few<MT, 1>(A, stream);
  if (ct == 2) return launch_few<MT, 2>(A, stream);
  if (ct == 3) return launch_few<MT, 3>(A, stream);
  if (ct == 5) return launch_few<MT, 5>(A, stream);
  return launch_few<MT, 9>(A, stream);
}

template <class X>
void launch_tiles(Mx4Args A, hipStream_t stream) {
  A.nbm = (int)((A.out.M + X::BM - 1) / X::BM);
  A.nbn = (int)((A.out.Ncols + X::BN - 1) / X::BN);
  hipLaunchKernelGGL((project_mx4_kernel<X>), dim3((unsigned)((int64_t)A.nbm * A.nbn)),
                     dim3(X::kThreads), 0, stream, A);
}

// Which kernel, and how many columns a few-token workgroup takes: by the cost
// of each in ns, as measured, with G turns or stages of 128 columns.
//
// Few tokens: the compute units work through their workgroups side by side, so
// a call lasts as long as the unit with the most of them.  A workgroup costs 31
// for each of its CT + MT fragments and turn (a single token's fragment, the
// same bytes on every lane, next to nothing) and 200 for each block it adds up;
// the CT of least cost over the rounds was within 5% of the best of CT = 1..9
// at 1, 16, 32 and 64 tokens x 16904 and 33808 columns.  64 tokens at d_model
// 8192 x 16904 columns: 22 us with CT = 5 (one round), 38 with 4 (two), 62 with
// 1.  CT = 9 leaves a unit one workgroup of four wavefronts, so it is for one
// block of tokens.
//
// Tiles: a round of 256 x 256 takes 7500 + 870 G; a unit holds two 128 x 128
// tiles, which take 5000 + 720 G together and 4000 + 330 G alone, so that they
// win where the larger tiles leave units idle or a last round nearly empty.
// us in few, 128 and 256: d_model 4096 x 4228 columns, 128 tokens 10, 13, 26;
// 512 tokens 26, 15, 28; 2048 tokens -, 39, 33.  d_model 8192 x 16904, 128
// tokens 37, 25, 47; 384 tokens 64, 51, 53; 768 tokens -, 100, 65.  d_model
// 16384 x 33808, 64 tokens 79, 100, 101; 384 tokens -, 213, 235; 4096 tokens
// -, 1587, 1192.  d_model 640 x 546, 512 tokens 5, 6, 12; 4096 tokens 24, 8, 14.
enum { kPickTile256 = 0, kPickTile128 = -1 };  // else the columns CT of the few-token kernel

int pick_kernel(const Mx4Args& A) {
  const int64_t M = A.out.M, Ncols = A.out.Ncols, G = A.K / 128, cus = compute_units();
  const int MT = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const int64_t tokens = (M + 16 * MT - 1) / (16 * MT);
  const int64_t rounds = (project_blocks(M, Ncols) + cus - 1) / cus;
  int64_t best = rounds * (7500 + 870 * G);
  int pick = kPickTile256;
  const int64_t small = ((M + 127) / 128) * ((Ncols + 127) / 128);
  if (small <= kMaxStrideBlocks) {  // work-items of a launch: 32 bits
    const int64_t each = (small + cus - 1) / cus;
    const int64_t cost = each / 2 * (5000 + 720 * G) + each % 2 * (4000 + 330 * G);
    if (cost < best) best = cost, pick = kPickTile128;
  }
  for (int ct : {1, 2, 3, 5, 9}) {
    if (ct == 9 && tokens > 1) break;
    const int64_t wgs = (Ncols + 16 * ct - 1) / (16 * ct) * tokens;
    if (wgs > kMaxProjTiles - 8 * tokens) continue;  // of 512 threads, in eights of column blocks
    const int64_t each = (ct + (M == 1 ? 0 : MT)) * G * 31 + 200 * ct * MT;
    const int64_t cost = (wgs + cus - 1) / cus * each + 2200;
    if (cost < best) best = cost, pick = ct;
  }
  return pick;
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
  const int pick = pick_kernel(A);
  if (pick == kPickTile256)
    launch_tiles<Tile256>(A, stream);
  else if (pick == kPickTile128)
    launch_tiles<Tile128>(A, stream);
  else if (A.out.M <= 16)
    launch_few_columns<1>(A, pick, stream);
  else if (A.out.M <= 32)
    launch_few_columns<2>(A, pick, stream);
  else
    launch_few_columns<4>(A, pick, stream);
  return hipGetLastError();
}

}  // namespace sdm
