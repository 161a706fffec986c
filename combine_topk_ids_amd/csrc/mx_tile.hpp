// mx_tile.hpp -- the matrix-product engine of the experts' products with MX-FP4 weights:
// expert_tile.hpp's, with operands of four bits and the scaled matrix instruction.
//
// A step covers 256 values of the contraction: 128 bytes of an MX-FP4 row, 256 of an FP8
// row (two parts of 128 bytes).  The 16x16x128 instruction takes half a step.
//
// Lane l of it holds row l % 16 of an operand; with q = l / 16, an MX-FP4 lane holds the
// 32 values of one scale block, the q-th of the four, and that block's scale byte
// (one of four in a register, by opsel); an FP8 lane holds values 16q .. 16q+15 and
// 64+16q .. 64+16q+15.  (Checked on the card, with scales that differ from block to block.)
//
//   MX-FP4 rows: lane group q takes blocks 2q and 2q + 1 of the step, one in each half, so
//     that both their scale bytes come in one 16-bit read.  The instruction scales and adds to
//     the fp32 accumulator: nothing is left for the vector units.
//   FP8 rows: a half is a 128-value block of the rows, whose products go to a sum of their own
//     (the weights' scales applied); times the row's fp32 scale it is added up.
//
// Scales go to LDS like the operands, a step's 8 bytes of a row as two 4-byte words (two
// blocks' fp32 scales of an FP8 row are as many).  Where scale rows are no whole words (K % 128
// != 0: ODD) it is the three words that the 8 bytes touch.  A scale byte past its row's
// end must not be the next row's NaN: words past it are not loaded (zero: 2^-127, times
// zero codes), bytes of a word past it are cleared after the read.
#pragma once

#include "expert_tile.hpp"

namespace moe {
namespace tile {

// As Shape.  FP8: the rows are FP8 (the weights are always MX-FP4).
template <int BI_, int BJ_, int WI_, int WJ_, int NST_, bool FP8_, bool ODD_, int WK_ = 1>
struct MxShape {
  static constexpr int BI = BI_, BJ = BJ_, WI = WI_, WJ = WJ_, NST = NST_, WK = WK_;
  static constexpr bool FP8 = FP8_, ODD = ODD_;
  static constexpr int kThreads = WI * WJ * kWave;
  static constexpr int FI = BI / WI / 16, FJ = BJ / WJ / 16;
  static constexpr int loads(int b) { return (b * 8 + kThreads - 1) / kThreads; }
  static constexpr int LI = loads(BI), LJ = loads(BJ), kParts = FP8 ? 2 : 1;
  static constexpr int kLoadRows = kThreads / 8;
  static constexpr int kBytesPart = LI * kThreads * 16;  // of I: 128 bytes of each row
  static constexpr int kBytesI = kParts * kBytesPart, kBytesJ = LJ * kThreads * 16;
  static constexpr int kWords = ODD ? 3 : 2;  // of scales, a row and step
  static constexpr int scale_loads(int b) { return (b * kWords + kThreads - 1) / kThreads; }
  static constexpr int LSI = scale_loads(BI), LSJ = scale_loads(BJ);
  static constexpr int kBytesSI = LSI * kThreads * 4, kBytesSJ = LSJ * kThreads * 4;
  static constexpr int kStage = kBytesI + kBytesJ + kBytesSI + kBytesSJ;
  static constexpr int kWaveCols = BJ / WJ;
  static constexpr int kTurnCols = WK == 1 && kWaveCols > 32 ? 32 : kWaveCols;
  static constexpr int kGroupLds = NST * kStage + WI * WJ * 16 * kTurnCols * 4;
  static constexpr int kLdsBytes = WK * kGroupLds;
  static constexpr int kByLds = 160 * 1024 / kLdsBytes, kByWaves = 8 / (WI * WJ * WK);
  static constexpr int kResident = kByLds < kByWaves ? kByLds : kByWaves;
  static constexpr int kWavesPerSimd = kResident * WI * WJ * WK >= 8 ? 2 : 1;
  static constexpr int kLoads = kParts * LI + LJ + LSI + LSJ;
  static_assert(!(FP8 && ODD), "FP8 rows have whole 128-value blocks");
  static_assert(BI % (16 * WI) == 0 && BJ % (16 * WJ) == 0, "whole blocks");
  static_assert(kLoads * (NST - 1) < 64, "the wait counter holds 63 loads");
  static_assert(kLdsBytes <= 160 * 1024, "LDS of a compute unit");
  static_assert(WK == 1 || (WI == 1 && WJ == 1 && FI == 1), "a group is one wave, its tile 16 rows");
};

// Scale rows of a tile (uniform).  `bytes` reach to the last row's end.
struct ScaleRows {
  const char *base;
  int bytes;
};

// A launch's lanes for the scales of B tile rows; ROW as in Along.
template <class S, int B, int N, class ROW>
struct WordLanes {
  ROW row;
  int row_bytes;
  __device__ __forceinline__ void init(int bytes) { row_bytes = bytes; }
  __device__ __forceinline__ void issue(lds_ptr to, const ScaleRows &s, int step) const {
    const int tid = group_thread<S>(), at = step * 8;
    to += group_wave<S>() * kWave * 4;
    // whole words from the one on that holds the first byte
    const int skip = S::ODD ? static_cast<int>(reinterpret_cast<uintptr_t>(s.base) & 3) : 0;
    const auto r = resource(s.base - skip + at, s.bytes == 0 ? 0 : max(((s.bytes + skip + 3) & ~3) - at, 0));
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = u * S::kThreads + tid;
      const int d = S::ODD ? i % 3 : i / B, tr = S::ODD ? i / 3 : i % B;
      const int start = static_cast<int>(row(tr)) * row_bytes + skip;
      const int word = (S::ODD ? start & ~3 : start) + d * 4;
      const bool in = (S::ODD ? tr < B : d < 2) && word + at < start + row_bytes;
      load_lds4(r, to + u * S::kThreads * 4, in ? static_cast<uint32_t>(word) : kNowhere);
    }
  }
};

struct MxSource {
  Operand i, j;
  ScaleRows x, w;
  int steps;
};
constexpr MxSource kNoMxSource{kNoOperand, kNoOperand, {nullptr, 0}, {nullptr, 0}, 0};
__device__ __forceinline__ MxSource either(bool c, const MxSource &a, const MxSource &b) {
  MxSource s = kNoMxSource;
  s.i = either(c, a.i, b.i);
  s.j = either(c, a.j, b.j);
  s.x = {c ? a.x.base : b.x.base, c ? a.x.bytes : b.x.bytes};
  s.w = {c ? a.w.base : b.w.base, c ? a.w.bytes : b.w.bytes};
  return s;
}

template <class S, class ROW>
struct MxFeed {
  Along<S, S::LI, SameRow> i;
  Along<S, S::LJ, ROW> j;
  WordLanes<S, S::BI, S::LSI, SameRow> x;
  WordLanes<S, S::BJ, S::LSJ, ROW> w;
  __device__ __forceinline__ void issue(lds_ptr lds, int stage, const MxSource &src, int step) const {
    lds_ptr to = lds + stage * S::kStage;
    if constexpr (S::WK > 1) step = step * S::WK + group_id<S>();
#pragma unroll
    for (int p = 0; p < S::kParts; ++p) i.issue(to + p * S::kBytesPart, src.i, step * S::kParts + p);
    j.issue(to + S::kBytesI, src.j, step);
    x.issue(to + S::kBytesI + S::kBytesJ, src.x, step);
    w.issue(to + S::kBytesI + S::kBytesJ + S::kBytesSI, src.w, step);
  }
};

// acc[a][b] = the products of cur's steps; as multiply() of expert_tile.hpp.
// skip_i, skip_j (ODD): what ScaleRows' first byte is past a whole word; blocks: scale blocks
// of a row.
template <class S, int FI, class F>
__device__ __forceinline__ void multiply_mx(lds_ptr lds, const F &feed, const MxSource &cur,
                                            const MxSource &next, int blocks, Progress &at,
                                            f32x4 (&acc)[FI][S::FJ]) {
  const Wave<S> w = this_wave<S>();
  const int lane = lane_id(), r = lane & 15, q = lane >> 4;
  // places in a stage: of the halves' chunks of row r of the wave's first block
  const int chunk = S::FP8 ? q : 2 * q;
  const int row_i = w.wi * 16 + r, row_j = w.wj * S::FJ * 16 + r;
  const int swap = S::FP8 ? 64 : 16;  // between the halves (of an FP8 part: between a lane's chunks)
  const int at_i = row_i * kStepBytes + ((chunk ^ (r & 7)) * 16);
  const int at_j = row_j * kStepBytes + ((chunk ^ (r & 7)) * 16);
  // and of their scales
  int scale_i, scale_j;
  if constexpr (S::FP8) {
    scale_i = row_i * 4;
    scale_j = row_j * 4 + q;
  } else if constexpr (S::ODD) {
    const int skip_i = static_cast<int>(reinterpret_cast<uintptr_t>(cur.x.base) & 3);
    const int skip_j = static_cast<int>(reinterpret_cast<uintptr_t>(cur.w.base) & 3);
    // (16 rows on, and an even number of gate rows on, a row starts at the same place in a word)
    scale_i = row_i * 12 + ((r * blocks + skip_i) & 3) + 2 * q;
    scale_j = row_j * 12 + ((r * blocks + skip_j) & 3) + 2 * q;
  } else {
    scale_i = (q >> 1) * S::BI * 4 + row_i * 4 + (q & 1) * 2;
    scale_j = (q >> 1) * S::BJ * 4 + row_j * 4 + (q & 1) * 2;
  }
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < S::FJ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = max(cur.steps, S::NST);
  int stage = at.stage;
  auto turn_over = [&](int t) {
    wait_behind<S::kLoads *(S::NST - 2)>(t < S::NST - 1 ? at.younger : 0);
    const int s = t + S::NST;
    const bool mine = s < steps;
    feed.issue(lds, stage, either(mine, cur, next), mine ? s : s - steps);
    stage = stage + 1 == S::NST ? 0 : stage + 1;
  };
  wait_behind<S::kLoads *(S::NST - 1)>(at.younger);

  i32x8 vi[2];
  i32x4 vj[S::FJ];
  float fi[2];                                      // FP8: the rows' scales
  int si[S::FP8 ? 1 : FI] = {}, sj[S::FJ];          // MX: both halves' bytes; FP8: one half's
  int mask = 0xFFFF;                                // ODD: of the step that si and sj belong to
  typedef uint16_t __attribute__((aligned(1), may_alias)) loose16;
  auto short_at = [&](lds_ptr p) -> int {
    if constexpr (S::ODD)
      return *(MOE_LDS const loose16 *)p & mask;
    else
      return *(MOE_LDS const uint16_t *)p;
  };
  // scale bytes that lie past the row's end in step t are cleared
  auto set_mask = [&](int t) {
    if constexpr (S::ODD) {
      if constexpr (S::WK > 1) t = t * S::WK + group_id<S>();
      const int left = blocks - t * 8 - 2 * q;
      mask = left >= 2 ? 0xFFFF : left == 1 ? 0xFF : 0;
    }
  };
  auto read_i = [&](int set, int blk, int half) {
    lds_ptr ti = lds + stage * S::kStage, ts = ti + S::kBytesI + S::kBytesJ;
    const int block = blk * S::WI * 16;
    if constexpr (S::FP8) {
      lds_ptr p = ti + half * S::kBytesPart + block * kStepBytes;
      vi[set] = __builtin_shufflevector(*(MOE_LDS const i32x4 *)(p + at_i), *(MOE_LDS const i32x4 *)(p + (at_i ^ 64)),
                                        0, 1, 2, 3, 4, 5, 6, 7);
      fi[set] = *(MOE_LDS const float *)(ts + scale_i + half * S::BI * 4 + block * 4);
    } else {
      const i32x4 v = *(MOE_LDS const i32x4 *)(ti + (half ? at_i ^ swap : at_i) + block * kStepBytes);
      vi[set] = __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
      if (half == 0) si[blk] = short_at(ts + scale_i + block * (S::ODD ? 12 : 4));
    }
  };
  auto read_j = [&](int b, int half) {
    lds_ptr tj = lds + stage * S::kStage + S::kBytesI, ts = tj + S::kBytesJ + S::kBytesSI;
    vj[b] = *(MOE_LDS const i32x4 *)(tj + (half ? at_j ^ swap : at_j) + b * 16 * kStepBytes);
    if constexpr (S::FP8)
      sj[b] = *(MOE_LDS const uint8_t *)(ts + scale_j + half * S::BJ * 4 + b * 16 * 4);
    else if (half == 0)
      sj[b] = short_at(ts + scale_j + b * 16 * (S::ODD ? 12 : 4));
  };
  auto wide = [](i32x4 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); };

  // A phase for each block of I in each half: its products run while the next block's rows are
  // read; in a half's last phase each block of J makes way, after its product, for
  // the next half's.
  auto half_step = [&](int t, auto which) {
    constexpr int H = decltype(which)::value;
#pragma unroll
    for (int a = 0; a < FI; ++a) {
      const int set = (H * FI + a) & 1;
      const bool last = a + 1 == FI;
      const int own = si[S::FP8 ? 0 : a];
      if (last && H == 1) {
        turn_over(t);
        set_mask(t + 1);
      }
      read_i(set ^ 1, last ? 0 : a + 1, last ? H ^ 1 : H);
      if constexpr (S::FP8) {
        // the product of block b, then what that of b - 1 adds to its sum
        f32x4 d[2];
#pragma unroll
        for (int b = 0; b <= S::FJ; ++b) {
          if (b < S::FJ) {
            d[b & 1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                wide(vj[b]), vi[set], f32x4{0.f, 0.f, 0.f, 0.f}, 4, 0, 0, sj[b], 0, 127);
            if (last) read_j(b, H ^ 1);
          }
          if (b > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[a][b - 1][i] = __builtin_fmaf(d[(b - 1) & 1][i], fi[set], acc[a][b - 1][i]);
          }
        }
      } else {
#pragma unroll
        for (int b = 0; b < S::FJ; ++b) {
          acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(vj[b]), vi[set], acc[a][b], 4, 4, H,
                                                                      sj[b], H, own);
          if (last) read_j(b, H ^ 1);
        }
      }
    }
  };
  set_mask(0);
#pragma unroll
  for (int b = 0; b < S::FJ; ++b) read_j(b, 0);
  read_i(0, 0, 0);
  for (int t = 0; t < steps; ++t) {
    half_step(t, std::integral_constant<int, 0>());
    half_step(t, std::integral_constant<int, 1>());
  }
  at.stage = stage;
}

}  // namespace tile
}  // namespace moe
