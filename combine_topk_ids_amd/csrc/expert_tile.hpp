// expert_tile.hpp -- the matrix-product engine of the experts' kernels
// (gfx950 MFMA): one workgroup computes a BI x BJ tile of
//
//   O[i][j] = sum_c I(i, c) * J(j, c),
//
// j contiguous in memory.  An operand is stored either "along c" (its rows
// are i or j, the contraction index is contiguous: token rows and weights of
// the forward products) or "across c" (its rows are the contraction index:
// the weights in the rows' gradient, both operands of the weights' gradient).
//
// J is the MFMA's A operand and I its B operand, so that a lane ends with four
// neighbouring j of one i, under one row scale.
//
// Memory path.  A step covers 128 bytes of the contraction (64 bf16 or 128 E4M3
// values).  Tiles go from global memory straight into LDS (16 bytes a lane, no
// registers), NST stages deep.  A workgroup takes tile after tile, and the
// loads run on across the tiles: the stage that a step has freed takes the loads
// of the step NST later, the next tile's first steps at a tile's end, so that
// memory is not idle while results leave.  One barrier a step both publishes a
// stage and frees the one before it.  Such a load writes 64
// consecutive 16-byte chunks of LDS, so there is no padding against bank conflicts;
// instead a lane picks which chunk of its row it fetches:
//   along c:  rows of 8 chunks, chunk c of row r at position c ^ (r & 7); the
//             16-byte operand reads of 8 consecutive lanes (8 rows, one chunk
//             index) then touch 8 different 16-byte bank groups;
//   across c: rows of 16-column groups (32 bytes), group g of row r at
//             g ^ f(r), f taking r's bits 0, 1, 3, 4: the 16 rows that one
//             transposing read visits for one group then lie in different banks.
// (Counters: no bank conflict in the bf16 products.)
// Where an operand ends, the buffer resource ends: loads past it fetch nothing and
// leave zeros in LDS.  What a lane adds to the resource's base is the same for
// every tile; a tile is a few scalars.
#pragma once

#include <type_traits>

#include "moe_device.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace tile {

#define MOE_LDS __attribute__((address_space(3)))

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef MOE_LDS char *lds_ptr;

constexpr int kStepBytes = 128;  // contraction bytes of one step
constexpr int kStepRows = 64;    // contraction rows of one step, stored across c
// An offset past every buffer resource used here (sizes stay below 2^31).
constexpr uint32_t kNowhere = 0x80000000u;
constexpr uint32_t kRecords = 0x7FFFFFFFu;

// WI x WJ waves; each owns FI x FJ blocks of 16 x 16.  XI/XJ: the operand is
// stored across c.  FP8: E4M3 codes (along c only) with block scales.  WK: such
// groups of waves in a workgroup; each takes every WK-th step through stages of its
// own, and the first adds up their sums (operands along c only).
template <int BI_, int BJ_, int WI_, int WJ_, int NST_, bool XI_ = false, bool XJ_ = false,
          bool FP8_ = false, int WK_ = 1>
struct Shape {
  static constexpr int BI = BI_, BJ = BJ_, WI = WI_, WJ = WJ_, NST = NST_, WK = WK_;
  static constexpr bool XI = XI_, XJ = XJ_, FP8 = FP8_;
  static constexpr int kThreads = WI * WJ * kWave;  // of a group; a workgroup has WK
  static constexpr int FI = BI / WI / 16, FJ = BJ / WJ / 16;
  // 16-byte loads a thread makes for an operand in a step; a tile smaller than one load
  // of every thread still gets a whole one (its spare rows are zeros)
  static constexpr int loads(int b) { return (b * 8 + kThreads - 1) / kThreads; }
  static constexpr int LI = loads(BI), LJ = loads(BJ);
  static constexpr int kLoadRows = kThreads / 8;  // tile rows between a thread's loads, along c
  static constexpr int kBytesI = LI * kThreads * 16, kBytesJ = LJ * kThreads * 16;
  static constexpr int kBytesScale = FP8 ? kThreads * 4 : 0;  // of each operand
  static constexpr int kStage = kBytesI + kBytesJ + 2 * kBytesScale;
  // the results' way out: see Transpose.  FP8's larger stages leave room for half
  static constexpr int kWaveCols = BJ / WJ;
  static constexpr int kTurnCols = FP8 && WK == 1 && kWaveCols > 32 ? 32 : kWaveCols;
  static constexpr int kGroupLds = NST * kStage + WI * WJ * 16 * kTurnCols * 4;
  static constexpr int kLdsBytes = WK * kGroupLds;
  // workgroups that a compute unit holds: LDS, and two waves a SIMD
  static constexpr int kByLds = 160 * 1024 / kLdsBytes, kByWaves = 8 / (WI * WJ * WK);
  static constexpr int kResident = kByLds < kByWaves ? kByLds : kByWaves;
  // Two waves a SIMD also keep the accumulators in the 256 registers that both
  // operands and results of an MFMA can name (with more, the compiler moves them to
  // and from the accumulation registers in the loop).  Small tiles with many
  // stages are held to one by their LDS.
  static constexpr int kWavesPerSimd = kResident * WI * WJ * WK >= 8 ? 2 : 1;
  static constexpr int kLoads = LI + LJ + (FP8 ? 2 : 0);  // of a wave and stage
  static_assert(BI % (16 * WI) == 0 && BJ % (16 * WJ) == 0, "whole blocks");
  static_assert(kLoads * (NST - 1) < 64, "the wait counter holds 63 loads");
  static_assert(kLdsBytes <= 160 * 1024, "LDS of a compute unit");
  static_assert(WK == 1 || (WI == 1 && WJ == 1 && FI == 1 && !XI && !XJ), "a group is one wave, its tile 16 rows");
};

// -------------------------------------------------------------- loaders ---

__device__ __forceinline__ int wave_id() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
}

// A group's number, and a thread's and wave's number within it.
template <class S>
__device__ __forceinline__ int group_id() {
  return S::WK == 1 ? 0 : wave_id() / (S::WI * S::WJ);
}
template <class S>
__device__ __forceinline__ int group_thread() {
  return S::WK == 1 ? threadIdx.x : threadIdx.x % S::kThreads;
}
template <class S>
__device__ __forceinline__ int group_wave() {
  return S::WK == 1 ? wave_id() : wave_id() % (S::WI * S::WJ);
}

// A buffer resource in the four scalar registers that an instruction names.
__device__ __forceinline__ i32x4 resource(const void *base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return i32x4{__builtin_amdgcn_readfirstlane(static_cast<int>(a)),
               __builtin_amdgcn_readfirstlane(static_cast<int>((a >> 32) & 0xFFFF)),
               __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), kRawBufferConfig};
}

// Loads straight into LDS: lane l's 16 (or 4) bytes go to `to` + 16 l (4 l); load u's
// to `to` + u * STRIDE.  Written as assembly because the compiler, which cannot
// tell the stages apart, otherwise waits for every such load in flight before each
// transposing read of LDS (seen in its output: the weights' gradient lost
// its prefetch to that).  These loads have no register results; what waits for them
// is wait_and_meet.  First line: scalars written by a vector instruction just before
// need five cycles; after a write of m0, one.
#define MOE_TO_LDS(N) \
  "s_add_u32 m0, m0, %[stride]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[o" #N "], %[r], 0 offen lds\n\t"
#define MOE_TO_LDS_FIRST \
  "s_nop 4\n\ts_mov_b32 m0, %[to]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[o0], %[r], 0 offen lds\n\t"
template <int STRIDE, int L>
__device__ __forceinline__ void load_lds16(i32x4 r, lds_ptr to, const uint32_t (&o)[L]) {
  static_assert(L == 1 || L == 2 || L == 4 || L == 8, "whole groups");
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<size_t>(to)));
  if constexpr (L == 1)
    asm volatile(MOE_TO_LDS_FIRST ::[o0] "v"(o[0]), [r] "s"(r), [to] "s"(at) : "memory", "m0", "scc");
  if constexpr (L == 2)
    asm volatile(MOE_TO_LDS_FIRST MOE_TO_LDS(1)::[o0] "v"(o[0]), [o1] "v"(o[1]), [r] "s"(r), [to] "s"(at),
                 [stride] "n"(STRIDE)
                 : "memory", "m0", "scc");
  if constexpr (L == 4)
    asm volatile(MOE_TO_LDS_FIRST MOE_TO_LDS(1) MOE_TO_LDS(2) MOE_TO_LDS(3)::[o0] "v"(o[0]), [o1] "v"(o[1]),
                 [o2] "v"(o[2]), [o3] "v"(o[3]), [r] "s"(r), [to] "s"(at), [stride] "n"(STRIDE)
                 : "memory", "m0", "scc");
  if constexpr (L == 8)
    asm volatile(MOE_TO_LDS_FIRST MOE_TO_LDS(1) MOE_TO_LDS(2) MOE_TO_LDS(3) MOE_TO_LDS(4) MOE_TO_LDS(5)
                     MOE_TO_LDS(6) MOE_TO_LDS(7)::[o0] "v"(o[0]), [o1] "v"(o[1]), [o2] "v"(o[2]),
                 [o3] "v"(o[3]), [o4] "v"(o[4]), [o5] "v"(o[5]), [o6] "v"(o[6]), [o7] "v"(o[7]), [r] "s"(r),
                 [to] "s"(at), [stride] "n"(STRIDE)
                 : "memory", "m0", "scc");
}
__device__ __forceinline__ void load_lds4(i32x4 r, lds_ptr to, uint32_t o) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<size_t>(to)));
  asm volatile("s_nop 4\n\ts_mov_b32 m0, %[to]\n\ts_nop 0\n\tbuffer_load_dword %[o], %[r], 0 offen lds" ::[o] "v"(o),
               [r] "s"(r), [to] "s"(at)
               : "memory", "m0");
}

// An operand of one tile (uniform).  Along c: `base` is its first row, `extent` the
// bytes up to the end of its last.  Across c: `base` is the first column's place
// in the first contraction row, `extent` the contraction rows, `skip` the bytes
// before that place in a row.
struct Operand {
  const char *base;
  int extent, skip;
};
constexpr Operand kNoOperand{nullptr, 0, 0};

// Rows of `row_bytes` stored along c.  ROW(r) maps a tile row to a row of the
// operand (it must satisfy ROW(a * kLoadRows + b) = ROW(a * kLoadRows) + ROW(b), b < kLoadRows).
template <class S, int L, class ROW>
struct Along {
  ROW row;
  int row_bytes, chunk;  // chunk: byte offset in a step of what this lane fetches
  uint32_t off;

  __device__ __forceinline__ void init(int bytes) {
    row_bytes = bytes;
    const int r = group_thread<S>() / 8;
    chunk = ((group_thread<S>() & 7) ^ (r & 7)) * 16;
    off = row(r) * bytes + chunk;
  }
  __device__ __forceinline__ void issue(lds_ptr to, const Operand &o, int step) const {
    const int at = step * kStepBytes;
    const uint32_t first = at + chunk < row_bytes ? off : kNowhere;  // the row's own end
    uint32_t place[L];
#pragma unroll
    for (int u = 0; u < L; ++u) place[u] = first + row(u * S::kLoadRows) * row_bytes;
    load_lds16<S::kThreads * 16>(resource(o.base + at, max(o.extent - at, 0)),
                                 to + group_wave<S>() * kWave * 16, place);
  }
};
struct SameRow {
  __device__ __forceinline__ uint32_t operator()(int r) const { return r; }
};

// The bank-spreading term of contraction row r in a tile of G 16-column groups.
template <int G>
__device__ __forceinline__ int group_mix(int r) {
  return ((r & 3) | (((r >> 3) & 3) << 2)) & (G - 1);
}

// Contraction rows of `ld` bytes, B columns of them.  Columns past the operand's
// are whatever follows in memory, inside the operand: they reach results past its
// columns only, which are not stored.
template <class S, int B, int L>
struct Across {
  static constexpr int kChunks = B / 8;                   // 16-byte chunks of a tile row
  static constexpr int kRows = S::kThreads / kChunks;     // rows between a thread's loads
  static_assert(kStepRows * kChunks == L * S::kThreads && kRows % 16 == 0, "whole loads");
  int ld;
  uint32_t off[2];  // of the even and of the odd loads, within their rows

  __device__ __forceinline__ void init(int row_bytes) {
    ld = row_bytes;
    const int ch = threadIdx.x % kChunks, r = threadIdx.x / kChunks;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      off[u] = r * ld + ((ch >> 1) ^ group_mix<B / 16>(u * kRows + r)) * 32 + (ch & 1) * 16;
  }
  __device__ __forceinline__ void issue(lds_ptr to, const Operand &o, int step) const {
    const int left = min(max(o.extent - step * kStepRows, 0), kStepRows);
    uint32_t place[L];
#pragma unroll
    for (int u = 0; u < L; ++u) place[u] = off[u & 1] + u * kRows * ld;
    load_lds16<S::kThreads * 16>(
        resource(o.base + static_cast<int64_t>(step) * kStepRows * ld, max(left * ld - o.skip, 0)),
        to + wave_id() * kWave * 16, place);
  }
};

// Block scales of an FP8 step: thread r fetches the scale of tile row r, and
// that of the weights' block r of the tile, `blocks` scales a row.
struct Scales {
  const float *base;
  int rows;  // scale rows from base on
};
template <class S>
struct ScaleLanes {
  int blocks;
  uint32_t row_off, weight_off;
  // weight_row: scale row of the weights' block that this thread fetches, relative to
  // the tile's first, or kNowhere
  __device__ __forceinline__ void init(int n, uint32_t weight_row) {
    blocks = n;
    row_off = group_thread<S>() < S::BI ? group_thread<S>() * n * 4 : kNowhere;
    weight_off = weight_row == kNowhere ? kNowhere : weight_row * n * 4;
  }
  __device__ __forceinline__ void issue(lds_ptr to, const Scales &x, const Scales &w, int step) const {
    to += group_wave<S>() * kWave * 4;
    load_lds4(resource(x.base + step, bytes(x, step)), to, row_off);
    load_lds4(resource(w.base + step, bytes(w, step)), to + S::kBytesScale, weight_off);
  }
  // left from the step's scales on; none past the last step, or of no tile
  __device__ __forceinline__ uint32_t bytes(const Scales &s, int step) const {
    return step < blocks ? max(s.rows * blocks - step, 0) * 4 : 0;
  }
};
struct NoScaleLanes {};  // bf16

// What a tile is fed from (uniform), and its steps.
struct Source {
  Operand i, j;
  Scales x, w;
  int steps;
};
constexpr Source kNoSource{kNoOperand, kNoOperand, {nullptr, 0}, {nullptr, 0}, 0};

// a or b, field by field (a choice between two whole ones would live in memory).
__device__ __forceinline__ Operand either(bool c, const Operand &a, const Operand &b) {
  return {c ? a.base : b.base, c ? a.extent : b.extent, c ? a.skip : b.skip};
}
template <bool FP8>
__device__ __forceinline__ Source either(bool c, const Source &a, const Source &b) {
  Source s = kNoSource;
  s.i = either(c, a.i, b.i);
  s.j = either(c, a.j, b.j);
  if constexpr (FP8) {
    s.x = {c ? a.x.base : b.x.base, c ? a.x.rows : b.x.rows};
    s.w = {c ? a.w.base : b.w.base, c ? a.w.rows : b.w.rows};
  }
  return s;
}

// A launch's lanes.
template <class S, class LI, class LJ, class LS>
struct Feed {
  LI i;
  LJ j;
  LS s;
  __device__ __forceinline__ void issue(lds_ptr lds, int stage, const Source &src, int step) const {
    lds_ptr to = lds + stage * S::kStage;
    if constexpr (S::WK > 1) step = step * S::WK + group_id<S>();
    i.issue(to, src.i, step);
    j.issue(to + S::kBytesI, src.j, step);
    if constexpr (S::FP8) s.issue(to + S::kBytesI + S::kBytesJ, src.x, src.w, step);
  }
};

// ------------------------------------------------------------- operands ---

// Where a lane finds its part of its wave's 16-row blocks in a stage: block b of
// the wave is block first + b * STRIDE of the tile.
template <int F, int B, int STRIDE, bool X>
struct Fragments;

template <int F, int B, int STRIDE>
struct Fragments<F, B, STRIDE, false> {
  int at[2];  // contraction halves of the step
  __device__ __forceinline__ void init(int first_block) {
    const int l = lane_id();
    at[0] = (first_block * 16 + (l & 15)) * kStepBytes + (((l >> 4) ^ (l & 7)) * 16);
    at[1] = at[0] ^ 64;
  }
  __device__ __forceinline__ i32x4 read(lds_ptr t, int b, int half) const {
    return *(MOE_LDS const i32x4 *)(t + at[half] + b * STRIDE * 16 * kStepBytes);
  }
};

template <int F, int B, int STRIDE>
struct Fragments<F, B, STRIDE, true> {
  int at[F];
  __device__ __forceinline__ void init(int first_block) {
    const int l = lane_id(), q = l >> 4, r = q * 8 + ((l >> 2) & 3);
#pragma unroll
    for (int b = 0; b < F; ++b)
      at[b] = r * B * 2 + ((first_block + b * STRIDE) ^ group_mix<B / 16>(r)) * 32 + (l & 3) * 8;
  }
  // two transposing reads: contraction rows 8q .. 8q+3 and 8q+4 .. 8q+7 of the half
  __device__ __forceinline__ i32x4 read(lds_ptr t, int b, int half) const {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    lds_ptr p = t + at[b] + half * 32 * B * 2;
    const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4 *)p));
    const i32x2 hi = __builtin_bit_cast(
        i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4 *)(p + 4 * B * 2)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
  }
};

// ------------------------------------------------------------ main loop ---

template <int N>
__device__ __forceinline__ void wait_and_meet() {
  // at most N of this wave's loads are outstanding and its LDS reads are done;
  // past the barrier that holds for every wave
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Order of half a step: an operand read, then some of its products, and so
// on.  Left alone, the compiler sinks each read to just before its use, to save
// registers, and waits for it there.
template <int READS, int PRODUCTS>
__device__ __forceinline__ void interleave() {
  constexpr int kEach = PRODUCTS / READS > 0 ? PRODUCTS / READS : 1;
#pragma unroll
  for (int i = 0; i < READS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      // LDS read
    __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);  // MFMA
  }
  __builtin_amdgcn_sched_group_barrier(0x008, PRODUCTS, 0);
  __builtin_amdgcn_sched_barrier(0);
}

template <class S>
struct Wave {
  int wi, wj;  // wi owns blocks wi, wi + WI, ... of I (so that a tile with few rows leaves
               // every wave the same share); wj a run of FJ blocks of J
};
template <class S>
__device__ __forceinline__ Wave<S> this_wave() {
  const int w = group_wave<S>();
  return {w / S::WJ, w % S::WJ};
}

// Where a wave stands between tiles.
struct Progress {
  int stage = 0;    // of the next tile's first step
  int younger = 0;  // stores it has issued after the next tile's first loads
};

// The loads of the first tile's first NST steps.
template <class S, class F>
__device__ __forceinline__ void start(lds_ptr lds, const F &feed, const Source &src) {
#pragma unroll
  for (int s = 0; s < S::NST; ++s) feed.issue(lds, s, src, s);
}

// Waits until at most N of this wave's loads, and the stores behind them, are
// outstanding, then for the other waves.  (The counter runs down in the order of
// issue, so a smaller count waits longer and is always safe.)
template <int N>
__device__ __forceinline__ void wait_behind(int stores) {
  if (stores >= 16)
    wait_and_meet<(N + 16 < 63 ? N + 16 : 63)>();
  else if (stores >= 8)
    wait_and_meet<(N + 8 < 63 ? N + 8 : 63)>();
  else
    wait_and_meet<N>();
}

// acc[a][b] = the products of cur's steps, for the wave's first FI blocks of I,
// while the loads run on into `next`.  On entry the loads of cur's first NST steps
// have been issued; on return those of next's.  scale_j(b): place of block b's
// scale among the stage's weight scales (FP8 only).
template <class S, int FI, class F, class ScaleJ>
__device__ __forceinline__ void multiply(lds_ptr lds, const F &feed, const Source &cur, const Source &next,
                                         Progress &at, ScaleJ scale_j, f32x4 (&acc)[FI][S::FJ]) {
  const Wave<S> w = this_wave<S>();
  Fragments<FI, S::BI, S::WI, S::XI> fi;
  Fragments<S::FJ, S::BJ, 1, S::XJ> fj;
  fi.init(w.wi);
  fj.init(w.wj * S::FJ);
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < S::FJ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  // (a shorter tile goes through NST steps all the same, of zeros)
  const int steps = max(cur.steps, S::NST);
  int stage = at.stage;
  // The next step's stage has landed, and every wave has read the last of this
  // one's, which takes the loads of step t + NST.
  auto turn_over = [&](int t) {
    wait_behind<S::kLoads *(S::NST - 2)>(t < S::NST - 1 ? at.younger : 0);
    const int s = t + S::NST;
    const bool mine = s < steps;
    feed.issue(lds, stage, either<S::FP8>(mine, cur, next), mine ? s : s - steps);
    stage = stage + 1 == S::NST ? 0 : stage + 1;
  };
  wait_behind<S::kLoads *(S::NST - 1)>(at.younger);

  if constexpr (S::FP8) {
    // What the sums keep.  The FP8 MFMA aligns the products of eight neighbouring columns to
    // the largest: with E the largest sum of the two codes' exponents among them (a
    // subnormal code's is -6), each is cut towards zero to a multiple of 2^(E-13), so
    // a group is off by less than 7 * 2^(E-13).  (Measured, for this form and the
    // 32-deep one.  A block of normal values: at most 2^-15 of the sum of magnitudes; h over
    // K = 7168, once rounded to bf16, differs from an fp32 evaluation by 2.8e-4, against 1.7e-3
    // for that rounding itself.)  Codes converted to bf16, which holds them exactly, would keep
    // 2^-23, at the bf16 rate (library products of 8192^3: 1457 TFLOP/s against 3150).  A
    // caller who takes FP8 operands has given up 2^-4 of each value for that rate, so the
    // FP8 instruction it is.  Past the block everything is fp32.
    //
    // A phase for each block of I: its products run while the next block's rows are
    // read.  In a step's last phase each block of J makes way, after its product,
    // for the next step's.
    i32x8 vi[2], vj[S::FJ];
    float si[2], sj[S::FJ];
    auto read_i = [&](int set, int blk) {
      lds_ptr ti = lds + stage * S::kStage, ts = ti + S::kBytesI + S::kBytesJ;
      vi[set] = __builtin_shufflevector(fi.read(ti, blk, 0), fi.read(ti, blk, 1), 0, 1, 2, 3, 4, 5, 6, 7);
      si[set] = *(MOE_LDS const float *)(ts + ((w.wi + blk * S::WI) * 16 + (lane_id() & 15)) * 4);
    };
    auto read_j = [&](int b) {
      lds_ptr tj = lds + stage * S::kStage + S::kBytesI, ts = tj + S::kBytesJ + S::kBytesScale;
      vj[b] = __builtin_shufflevector(fj.read(tj, b, 0), fj.read(tj, b, 1), 0, 1, 2, 3, 4, 5, 6, 7);
      sj[b] = *(MOE_LDS const float *)(ts + scale_j(b) * 4);
    };
    auto step = [&](int t, auto odd) {
#pragma unroll
      for (int a = 0; a < FI; ++a) {
        const int set = (a + (FI % 2 ? decltype(odd)::value : 0)) & 1;
        const bool last = a + 1 == FI;
        if (last) turn_over(t);
        read_i(set ^ 1, last ? 0 : a + 1);
        // the product of block b, then what that of b - 1 adds to its sum
        f32x4 d[2];
        float scale[2];
#pragma unroll
        for (int b = 0; b <= S::FJ; ++b) {
          if (b < S::FJ) {
            scale[b & 1] = si[set] * sj[b];
            d[b & 1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                vj[b], vi[set], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
            if (last) read_j(b);
          }
          if (b > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[a][b - 1][i] = __builtin_fmaf(d[(b - 1) & 1][i], scale[(b - 1) & 1], acc[a][b - 1][i]);
          }
        }
      }
    };
#pragma unroll
    for (int b = 0; b < S::FJ; ++b) read_j(b);
    read_i(0, 0);
    for (int t = 0; t < steps; t += 2) {
      step(t, std::integral_constant<int, 0>());
      if (t + 1 < steps) step(t + 1, std::integral_constant<int, 1>());
    }
  } else {
    // Operands are read half a step ahead of the products that use them, so
    // that the matrix cores have work while the next operands leave LDS.
    bf16x8 vi[2][FI], vj[2][S::FJ];
    auto read = [&](int half) {
      lds_ptr ti = lds + stage * S::kStage, tj = ti + S::kBytesI;
#pragma unroll
      for (int b = 0; b < S::FJ; ++b) vj[half][b] = __builtin_bit_cast(bf16x8, fj.read(tj, b, half));
#pragma unroll
      for (int a = 0; a < FI; ++a) vi[half][a] = __builtin_bit_cast(bf16x8, fi.read(ti, a, half));
    };
    auto products = [&](int half) {
#pragma unroll
      for (int a = 0; a < FI; ++a)
#pragma unroll
        for (int b = 0; b < S::FJ; ++b)
          acc[a][b] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(vj[half][b], vi[half][a], acc[a][b], 0, 0, 0);
      // transposing reads come in twos
      interleave<FI * (S::XI ? 2 : 1) + S::FJ * (S::XJ ? 2 : 1), FI * S::FJ>();
    };
    read(0);
    for (int t = 0; t < steps; ++t) {
      read(1);
      products(0);
      turn_over(t);
      read(0);
      products(1);
    }
  }
  at.stage = stage;
}

// ------------------------------------------------------------- epilogue ---

// The lane number, as a value the compiler cannot compute ahead: what the
// epilogue derives from it is then not kept in registers through the main loop.
__device__ __forceinline__ int late_lane_id() {
  int l = lane_id();
  asm volatile("" : "+v"(l));
  return l;
}

// A wave's results leave through LDS: block row a (16 rows of I) of COLS columns,
// fp32, is written as the MFMA leaves it (4 columns of one row a lane) and read
// back as 8 columns of one row a lane, so that global rows are read and written
// in 16-byte pieces of whole lines.  The 16-byte chunk c of row r lies at c ^ r:
// neither direction has bank conflicts.  One wave's region is its own: LDS
// operations of a wave complete in order, so no barrier is needed.
template <int COLS>
struct Transpose {
  // of this wave, behind the stages
  template <class S>
  __device__ __forceinline__ static Transpose make(lds_ptr lds, int lane) {
    return {lds + S::NST * S::kStage + group_wave<S>() * kBytes, lane};
  }
  static constexpr int kChunks = COLS / 4;
  static constexpr int kBytes = 16 * COLS * 4;
  static constexpr int kLanesPerRow = COLS / 8;
  static constexpr int kPasses = 16 * kLanesPerRow / kWave;  // rows a lane gets back
  static_assert(kPasses >= 1, "at least 32 columns");
  lds_ptr base;
  int l;  // the lane
  __device__ __forceinline__ void put(int b, const f32x4 v) const {  // columns 16b .. 16b+15
    const int r = l & 15, c = b * 4 + (l >> 4);
    *(MOE_LDS f32x4 *)(base + r * COLS * 4 + ((c ^ r) & (kChunks - 1)) * 16) = v;
  }
  __device__ __forceinline__ int row(int pass) const {
    return pass * (kWave / kLanesPerRow) + l / kLanesPerRow;
  }
  __device__ __forceinline__ int col() const { return l % kLanesPerRow * 8; }
  __device__ __forceinline__ void get(int pass, float (&v)[8]) const {
    const int r = row(pass), c = col() / 4;
    const f32x4 a = *(MOE_LDS const f32x4 *)(base + r * COLS * 4 + ((c ^ r) & (kChunks - 1)) * 16);
    const f32x4 b = *(MOE_LDS const f32x4 *)(base + r * COLS * 4 + (((c + 1) ^ r) & (kChunks - 1)) * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
};

__device__ __forceinline__ bf16x8 round8(const float (&v)[8]) {
  bf16x8 r;
#pragma unroll
  for (int c = 0; c < 8; ++c) r[c] = static_cast<__bf16>(v[c]);
  return r;
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8]) {
  *reinterpret_cast<bf16x8 *>(p) = round8(v);
}
// Through a buffer resource, at byte `off`; kNowhere drops it.  POLICY: cache bits.
// Always one store of the wave, whichever lanes have something to store
// (wait_behind counts them).
template <int POLICY = kLoadDefault>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[8]) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, round8(v)), r, static_cast<int>(off), 0,
                                         POLICY);
}

__device__ __forceinline__ void store8_f32(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[8]) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const f32x4 lo{v[0], v[1], v[2], v[3]}, hi{v[4], v[5], v[6], v[7]};
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, lo), r, static_cast<int>(off), 0, 0);
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, hi), r, static_cast<int>(off), 16, 0);
}

// ---------------------------------------------------------- expert rows ---

// Rows of expert e that hold a token, whatever the plan's arrays hold:
// start + count stays within `rows`.
struct ExpertRows {
  int start, count;
};
__device__ __forceinline__ ExpertRows expert_rows(const int32_t *offsets, const int32_t *counts, int e,
                                                  int rows) {
  const int a = offsets[e], b = offsets[e + 1];
  ExpertRows r;
  r.start = min(max(a, 0), rows);
  const int64_t room = static_cast<int64_t>(b) - a;  // the fixed capacity may be less than the count
  int64_t n = counts[e];
  n = n < room ? n : room;
  n = n < rows - r.start ? n : rows - r.start;
  r.count = n > 0 ? static_cast<int>(n) : 0;
  return r;
}

struct RowTile {
  int e;             // expert, -1: no tile
  int start, count;  // its rows
  int i0, j;         // first row of the tile in the expert, column tile
};

// Row tiles are handed out expert by expert, groups of 8 row tiles at a time,
// every column tile of a group before the next; neighbours in this order share
// an expert's weights and rows.  Workgroups go round the 8 XCDs in turn, so an
// XCD takes one contiguous run of the order and its workgroups walk through it
// side by side: its L2 sees each panel once.
template <int BI>
struct RowTiles {
  const int32_t *offsets, *counts;
  int n_experts, rows, col_tiles;
  int per;          // experts a lane adds up (at most 16)
  int incl, mine;   // row tiles of the lanes up to this one, and of this one
  int64_t total, chunk;

  __device__ __forceinline__ void init(const int32_t *off, const int32_t *cnt, int experts, int nrows,
                                       int cols) {
    offsets = off;
    counts = cnt;
    n_experts = experts;
    rows = nrows;
    col_tiles = cols;
    per = (n_experts + kWave - 1) / kWave;
    mine = 0;
    for (int u = 0; u < per; ++u) {
      const int e = lane_id() * per + u;
      if (e < n_experts) mine += min((expert_rows(offsets, counts, e, rows).count + BI - 1) / BI, 1 << 24);
    }
    // (2^24 row tiles are more than any routing within check_expert_op's limits has; plan
    // arrays that describe none cannot make the sums below overflow)
    mine = min(mine, 1 << 24);
    incl = wave_incl_scan(mine);
    total = static_cast<int64_t>(__builtin_amdgcn_readlane(incl, kWave - 1)) * col_tiles;
    chunk = (total + 7) / 8;
  }

  // The i-th tile of this workgroup.  An expert's last row tile holds fewer rows and
  // takes less time; the workgroups change places from round to round, so that
  // none meets such tiles every time.
  __device__ __forceinline__ RowTile find(int i) const {
    RowTile r;
    r.e = -1;
    const int each = gridDim.x / 8;  // workgroups of an XCD
    const int64_t pos = static_cast<int64_t>(i) * each + (blockIdx.x / 8 + i) % each;
    const int64_t t = (blockIdx.x % 8) * chunk + pos;
    // (past the end in one round is past it in every later one)
    if (pos >= chunk || t >= total) return r;
    const uint64_t past = ballot(static_cast<int64_t>(incl) * col_tiles > t);
    if (past == 0) return r;
    const int owner = __builtin_ctzll(past);
    int before = __builtin_amdgcn_readlane(incl - mine, owner);
    // the owner's experts, one per lane
    const int lane = lane_id(), e = owner * per + lane;
    ExpertRows x{0, 0};
    if (lane < per && e < n_experts) x = expert_rows(offsets, counts, e, rows);
    const int tiles = (x.count + BI - 1) / BI;
    const int upto = wave_incl_scan(tiles);
    const uint64_t here = ballot(static_cast<int64_t>(before + upto) * col_tiles > t);
    if (here == 0) return r;  // the plan changed since init()
    const int who = __builtin_ctzll(here);
    r.e = owner * per + who;
    r.start = __builtin_amdgcn_readlane(x.start, who);
    r.count = __builtin_amdgcn_readlane(x.count, who);
    const int ti = __builtin_amdgcn_readlane(tiles, who);
    before += __builtin_amdgcn_readlane(upto - tiles, who);
    const int q = static_cast<int>(t - static_cast<int64_t>(before) * col_tiles);
    const int group = q / (8 * col_tiles), rest = q - group * 8 * col_tiles;
    const int size = min(8, ti - group * 8);
    r.j = rest / size;
    r.i0 = (group * 8 + rest - r.j * size) * BI;
    return r;
  }
};

// f(integral_constant<int, FI>) with the blocks of I that each wave needs for a tile
// of `rows` rows, in quarters of all of them.
template <class S, class F>
__device__ __forceinline__ void with_blocks(int rows, F f) {
  if constexpr (S::FI % 4 == 0) {
    const int quarters = (rows + S::BI / 4 - 1) / (S::BI / 4);
    if (quarters == 1) return f(std::integral_constant<int, S::FI / 4>());
    if (quarters == 2) return f(std::integral_constant<int, S::FI / 2>());
    if (quarters == 3) return f(std::integral_constant<int, S::FI / 4 * 3>());
  }
  f(std::integral_constant<int, S::FI>());
}

constexpr int kComputeUnits = 256;

// Tiles of B columns that cover n of them.
template <int B>
inline int64_t col_tiles(int n) {
  return (n + B - 1) / B;
}

// Fewer tiles than this leave so many of the 256 compute units without work that
// smaller tiles are faster, though each feeds the matrix cores less well.  (Rows'
// gradient, K = 2N = 1024: 8 experts of 512 rows, 160 tiles of 256 x 256, 51.9 us, of
// 128 x 128, 52.4; of 256 rows, 64 tiles, 46.3 against 23.4; of 128 rows, 127
// tiles of 128 x 128, 22.5 against 16.8 of 64 x 128.)
constexpr int kEnoughTiles = 128;

// Workgroups of a launch: at most `resident` a compute unit, which then take tile
// after tile, or as many as there are tiles (kAnyNumber); a multiple of the 8 XCDs.
constexpr int kAnyNumber = 1 << 20;
inline uint32_t tile_grid(int64_t tiles, int resident) {
  const int64_t most = static_cast<int64_t>(kComputeUnits) * resident;
  return static_cast<uint32_t>(((tiles < most ? tiles : most) + 7) / 8 * 8);
}

// Workgroups that cover every row tile of any routing of at most `pairs` rows.
template <int BI>
inline int64_t row_tile_bound(int64_t pairs, int n_experts) {
  const int64_t used = pairs < n_experts ? pairs : n_experts;
  return (pairs + used * (BI - 1)) / BI;
}

// ---------------------------------------------------------- activations ---

// The hardware's exp2 and reciprocal, a unit in the last place each: off by (|z| + 8) 2^-23
// of its value, which the rounding to bf16 hides.  Below 2^-126 it is zero: an
// activation of z < -87 comes out as -0 where its value is less than |z| 2^-126.
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// value and slope of an activation (a moe_act)
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == MOE_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == MOE_ACT_GELU_TANH)  // (1 + tanh a) / 2 = sigmoid(2a)
    return z * sigmoid(1.5957691216057308f * (z + 0.044715f * z * z * z));
  if constexpr (ACT == MOE_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  return z;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoid(z);
    return s * (1.0f + z * (1.0f - s));
  }
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    // sigmoid' has left the fp32 range of 1 long before; z * z could overflow
    if (fabsf(z) > 16.0f) return z > 0.0f ? 1.0f : 0.0f;
    const float s = sigmoid(1.5957691216057308f * (z + 0.044715f * z * z * z));
    return s + z * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * z * z);
  }
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  return 1.0f;
}

// f(integral_constant<ACT>) for a runtime activation
template <class F>
inline hipError_t with_act(int act, F f) {
  switch (act) {
    case MOE_ACT_SILU: return f(std::integral_constant<int, MOE_ACT_SILU>());
    case MOE_ACT_GELU_TANH: return f(std::integral_constant<int, MOE_ACT_GELU_TANH>());
    case MOE_ACT_RELU: return f(std::integral_constant<int, MOE_ACT_RELU>());
    default: return f(std::integral_constant<int, MOE_ACT_NONE>());
  }
}

}  // namespace tile
}  // namespace moe
