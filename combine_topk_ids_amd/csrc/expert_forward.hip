// expert_forward.hip -- the experts' forward products over the packed rows:
//
//   gated block   z = x w_e^T + b_e (2F columns),  h = act(z[:F]) * z[F:]
//   linear layer  z = x w_e^T + b_e,               y = act(z) + residual
//
// bf16: every sum is an fp32 MFMA accumulator.  FP8: the matrix instruction adds the 128
// products of a scale block and keeps fewer bits of the small ones (expert_tile.hpp says
// which, and why it is used); the blocks' sums are scaled and added in fp32.  z, h and y
// are rounded once, to bf16, when they are stored (the activation sees the unrounded z).
#include "expert_tile.hpp"

namespace moe {
namespace {

using namespace tile;

struct ForwardArgs {
  const void *x, *w;
  const float *x_scales, *w_scales, *bias;
  const uint16_t *residual;
  uint16_t *y, *preact;
  const int32_t *offsets, *counts;
  int n_experts, rows;
  int k, n;       // columns of a row of x; columns of y
  int col_tiles;
};

// GLU: a tile holds BJ / 2 columns of h; its weight rows go to LDS as
// alternating 16-row blocks of gate and up rows, so that a wave holds both
// halves of each of its columns and the product is formed in registers.
struct GateUpRow {
  int n;
  __device__ __forceinline__ uint32_t operator()(int r) const {
    return (r & 16 ? n : 0) + (r >> 5) * 16 + (r & 15);
  }
};

template <class S, bool GLU, int ACT>
__global__ __launch_bounds__(S::kThreads *S::WK, S::kWavesPerSimd) void forward_kernel(ForwardArgs g) {
  __shared__ __align__(1024) char smem[S::kLdsBytes];
  lds_ptr lds = (lds_ptr)smem + group_id<S>() * S::kGroupLds;
  constexpr int kSize = S::FP8 ? 1 : 2;
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;  // columns of y in a tile
  constexpr int kWaveCols = kCols / S::WJ;        // and in a wave
  const int row_bytes = g.k * kSize, wrows = GLU ? 2 * g.n : g.n, blocks = g.k / 128;
  const Wave<S> w = this_wave<S>();
  RowTiles<S::BI> order;
  order.init(g.offsets, g.counts, g.n_experts, g.rows, g.col_tiles);
  RowTile t = order.find(0);
  if (t.e < 0) return;

  typedef typename std::conditional<GLU, GateUpRow, SameRow>::type WeightRow;
  typedef typename std::conditional<S::FP8, ScaleLanes<S>, NoScaleLanes>::type ScaleLane;
  Feed<S, Along<S, S::LI, SameRow>, Along<S, S::LJ, WeightRow>, ScaleLane> feed;
  feed.i.init(row_bytes);
  if constexpr (GLU) feed.j.row.n = g.n;
  feed.j.init(row_bytes);
  if constexpr (S::FP8) {
    // the scales of a tile's weights: its gate and its up block, or its
    // 128-column blocks
    const int tid = group_thread<S>();
    feed.s.init(blocks, tid < (GLU ? 2 : (S::BJ + 127) / 128) ? (GLU ? tid * (g.n / 128) : tid) : kNowhere);
  }
  auto source = [&](const RowTile &r) {
    if (r.e < 0) return kNoSource;
    const int j0 = r.j * kCols, left = min(r.count - r.i0, S::BI);
    const int64_t row0 = static_cast<int64_t>(r.start) + r.i0, wrow0 = static_cast<int64_t>(r.e) * wrows + j0;
    Source s = kNoSource;
    s.i = {static_cast<const char *>(g.x) + row0 * row_bytes, left * row_bytes, 0};
    s.j = {static_cast<const char *>(g.w) + wrow0 * row_bytes, (wrows - j0) * row_bytes, 0};
    if constexpr (S::FP8) {
      s.x = {g.x_scales + row0 * blocks, left};
      s.w = {g.w_scales + (static_cast<int64_t>(r.e) * (wrows / 128) + j0 / 128) * blocks,
             wrows / 128 - j0 / 128};
    }
    s.steps = (row_bytes + kStepBytes * S::WK - 1) / (kStepBytes * S::WK);
    return s;
  };
  auto scale_j = [&](int b) { return GLU ? b & 1 : (w.wj * S::FJ + b) * 16 / 128; };

  Source cur = source(t), following;
  start<S>(lds, feed, cur);
  Progress at;
  auto one_tile = [&](auto own_blocks) {
    constexpr int FI = decltype(own_blocks)::value;
    constexpr int kTurnCols = GLU ? kWaveCols : S::kTurnCols, kTurns = kWaveCols / kTurnCols;
    constexpr int kTurnBlocks = kTurnCols / 16;
    f32x4 acc[FI][S::FJ];
    multiply<S, FI>(lds, feed, cur, following, at, scale_j, acc);
    const int lane = late_lane_id();
    if constexpr (S::WK > 1) {
      // the groups' sums, added in order by the first, through what is its way out
      lds_ptr sums = lds + S::NST * S::kStage + lane * 16;
      if (group_id<S>() > 0) {
#pragma unroll
        for (int b = 0; b < S::FJ; ++b) *(MOE_LDS f32x4 *)(sums + b * kWave * 16) = acc[0][b];
      }
      __syncthreads();
      if (group_id<S>() > 0) {
        at.younger = 0;
        return;
      }
#pragma unroll
      for (int q = 1; q < S::WK; ++q)
#pragma unroll
        for (int b = 0; b < S::FJ; ++b)
          acc[0][b] += *(MOE_LDS const f32x4 *)(sums + q * S::kGroupLds + b * kWave * 16);
    }
    const auto turn = Transpose<kTurnCols>::template make<S>(lds, lane);
    const float *bias = g.bias ? g.bias + static_cast<int64_t>(t.e) * wrows : nullptr;
    const int col0 = t.j * kCols + w.wj * kWaveCols;  // of the wave
    const int left = t.count - t.i0;                  // rows of the tile
    const int64_t row0 = static_cast<int64_t>(t.start) + t.i0;
    f32x4 shift[S::FJ];
#pragma unroll
    for (int b = 0; b < S::FJ; ++b) {
      const int c = col0 + (GLU ? b / 2 : b) * 16 + (lane >> 4) * 4;
      shift[b] = bias && c < g.n ? *reinterpret_cast<const f32x4 *>(bias + (GLU && b % 2 ? g.n : 0) + c)
                                 : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // byte offset in rows of `ld` columns of what pass p of block row a holds
    auto place = [&](int a, int p, int h, int ld) {
      const int i = (w.wi + a * S::WI) * 16 + turn.row(p), col = col0 + h * kTurnCols + turn.col();
      return i < left && col < g.n ? static_cast<uint32_t>(i * ld + col) * 2 : kNowhere;
    };
    // all of the residual before the first store: one trip to memory
    uint4 add[GLU ? 1 : FI][kTurns][turn.kPasses];
    if constexpr (!GLU) {
      if (g.residual) {
        const auto r = buffer_rsrc(g.residual + row0 * g.n, kRecords);
#pragma unroll
        for (int a = 0; a < FI; ++a)
#pragma unroll
          for (int h = 0; h < kTurns; ++h)
#pragma unroll
            for (int p = 0; p < turn.kPasses; ++p)
              add[a][h][p] = __builtin_bit_cast(
                  uint4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(place(a, p, h, g.n)), 0,
                                                               kLoadDefault));
      }
    }
#pragma unroll
    for (int a = 0; a < FI; ++a) {
      // what turn holds, to rows of `ld` columns from `to`
      auto leave = [&](uint16_t *to, int ld, int h, bool residual) {
        const auto r = buffer_rsrc(to + row0 * ld, kRecords);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int p = 0; p < turn.kPasses; ++p) {
          float v[8];
          turn.get(p, v);
          if constexpr (!GLU) {
            if (residual) {
              float more[8];
              unpack8(add[a][h][p], more);
#pragma unroll
              for (int c = 0; c < 8; ++c) v[c] += more[c];
            }
          }
          store8(r, place(a, p, h, ld), v);
        }
        __builtin_amdgcn_wave_barrier();
      };
#pragma unroll
      for (int b = 0; b < S::FJ; ++b) acc[a][b] += shift[b];
      if (g.preact) {
        constexpr int kParts = GLU ? 2 : 1;
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int h = 0; h < kTurns; ++h) {
#pragma unroll
            for (int b = 0; b < kTurnBlocks; ++b)
              turn.put(b, acc[a][(h * kTurnBlocks + b) * kParts + part]);
            leave(g.preact + part * g.n, wrows, h, false);
          }
      }
#pragma unroll
      for (int h = 0; h < kTurns; ++h) {
#pragma unroll
        for (int b = 0; b < kTurnBlocks; ++b) {
          const int at_b = (h * kTurnBlocks + b) * (GLU ? 2 : 1);
          f32x4 y;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            y[c] = act_value<ACT>(acc[a][at_b][c]) * (GLU ? acc[a][at_b + (GLU ? 1 : 0)][c] : 1.0f);
          turn.put(b, y);
        }
        leave(g.y, g.n, h, g.residual != nullptr);
      }
    }
    at.younger = FI * kTurns * turn.kPasses;
  };
  for (int n = 1; t.e >= 0; ++n) {
    const RowTile next = order.find(n);
    following = source(next);
    with_blocks<S>(t.count - t.i0, one_tile);
    t = next;
    cur = following;
  }
  wait_and_meet<0>();  // loads past the last tile fetch nothing, but write LDS
}

// resident: tile_grid's
template <class S, bool GLU>
hipError_t launch(ForwardArgs g, int64_t pairs, int act, hipStream_t stream, int resident = S::kResident) {
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;
  g.col_tiles = (g.n + kCols - 1) / kCols;
  const int64_t tiles = row_tile_bound<S::BI>(pairs, g.n_experts) * g.col_tiles;
  const uint32_t grid = tile_grid(tiles, resident);
  return with_act(act, [&](auto a) {
    forward_kernel<S, GLU, decltype(a)::value><<<grid, S::kThreads * S::WK, 0, stream>>>(g);
    return hipGetLastError();
  });
}

// Which tile, by the rows an expert has on average and by whether larger tiles would
// leave compute units without work.  Measured at K = 4096, F = 1024 (gated, 64
// experts, top 6; us a call, bf16 unless FP8 is said):
//   rows an expert       0.1     0.75    4      64     96    128    192
//   16 x 64, K in four   18.2   105.6  178.4   393.9
//   16 x 64              21.2   115.5  187.1   420.6  586.1  748.8 1038.9
//   128 x 128            54.0   145.0  181.9   192.6  205.8  310.8  315.8
//   256 x 256            72.3   165.6  193.3   211.1  224.2  235.6  268.9
// A long contraction is split over the four waves of a 16 x 64 tile, for few rows an
// expert (12 rows: 181.0 against 181.9 of 128 x 128, FP8 102.6 against 124.2; 16:
// 192.2 against 181.9) and for few tiles, whose time is that of one chain of steps
// (1 expert of 40 rows, K = 4096, F = 512: 10.5 against 23.3; 512 tiles, K = 7168:
// 29.3 against 38.7; 528 tiles, K = 2048: 16.9 against 14.3).  A short one is not
// worth the join (linear, 64 experts of 1 row, K = 2048: 120.4 against 125.0; K = 1024,
// 0.4 rows: 38.9 against 36.8).
// The rows an expert has on average are all the host knows.  Where the routing sends
// them all to a few experts, the tile picked for few rows is the wrong one (K = 4096,
// F = 1024, bf16; 64 experts, 768 rows on six of them: K in four 50 us, 64 x 128
// 25, 128 x 128 42; 256 experts, 512 rows on each of six: 182, 69, 54; 6144 rows of 64 experts
// on six: 128 x 128 97, 256 x 256 96).
// FP8 stays with 128 x 128: a 256 x 256 tile's sums, operands and block products
// do not fit the registers.  With many rows its workgroups take one tile each, so that
// tiles which share weights start together: that pays for the largest weights and a
// long contraction, and costs the run-on of the loads, and so time, elsewhere (gated, us,
// one tile each against tile after tile; F = 2048, 256 rows an expert):
//   K                 1024         2048         4096          7168
//   8 experts      17.2 / 17.8  26.7 / 26.8  49.0 / 49.1   79.7 / 78.4
//   64 experts      128 / 115    216 / 197    404 / 379     694 / 678
//   256 experts     534 / 438    882 / 780   1563 / 1561   2748 / 3107
// (L2 misses of the last: 15.2 GB against 22.9.)  With few rows the weights pass
// once in any order (1295 against 1204 us at 4 rows).
template <bool GLU, bool FP8>
hipError_t launch_sized(const ForwardArgs &g, int64_t pairs, int act, hipStream_t stream) {
  typedef Shape<16, 64, 1, 1, 3, false, false, FP8, 4> Split;
  typedef Shape<16, 64, 1, 1, 6, false, false, FP8> Few;
  typedef Shape<64, 128, 2, 2, 3, false, false, FP8> Low;
  typedef Shape<128, 128, 2, 2, 2, false, false, FP8> Some;
  const int64_t used = pairs < g.n_experts ? pairs : g.n_experts, rows = (pairs + used - 1) / used;
  const int wrows = g.n * (GLU ? 2 : 1);
  const int64_t tiles = row_tile_bound<Some::BI>(pairs, g.n_experts) * col_tiles<Some::BJ>(wrows);
  const int64_t split_tiles = row_tile_bound<Split::BI>(pairs, g.n_experts) * col_tiles<Split::BJ>(wrows);
  if (g.k >= 2048 && (rows <= 12 || split_tiles <= 2 * kComputeUnits))
    return launch<Split, GLU>(g, pairs, act, stream);
  if (rows <= 16 && tiles < 4 * kComputeUnits) return launch<Few, GLU>(g, pairs, act, stream);
  if (tiles < kEnoughTiles) return launch<Low, GLU>(g, pairs, act, stream);
  if (rows <= 112) return launch<Some, GLU>(g, pairs, act, stream);
  if constexpr (FP8) {
    return launch<Some, GLU>(g, pairs, act, stream, kAnyNumber);
  } else {
    typedef Shape<256, 256, 2, 4, 2> Many;
    if (row_tile_bound<Many::BI>(pairs, g.n_experts) * col_tiles<Many::BJ>(wrows) < kEnoughTiles)
      return launch<Some, GLU>(g, pairs, act, stream);
    return launch<Many, GLU>(g, pairs, act, stream);
  }
}

}  // namespace

hipError_t launch_expert_forward(const moe_problem &p, const moe_plan &plan, const moe_expert_op &op,
                                 bool glu, const ExpertForward &f, hipStream_t stream) {
  const int64_t rows = max_rows(p), pairs = expert_row_bound(p);
  if (pairs == 0) return hipSuccess;
  ForwardArgs g;
  g.x = f.x;
  g.w = f.w;
  g.x_scales = f.x_scales;
  g.w_scales = f.w_scales;
  g.bias = f.bias;
  g.residual = f.residual;
  g.y = f.y;
  g.preact = f.preact;
  g.offsets = plan.expert_offsets;
  g.counts = plan.expert_counts;
  g.n_experts = p.n_experts;
  g.rows = static_cast<int>(rows);
  g.k = op.in_dim;
  g.n = op.out_dim;
  const bool fp8 = op.fmt == MOE_FMT_FP8_E4M3_B128;
  if (glu)
    return fp8 ? launch_sized<true, true>(g, pairs, op.act, stream)
               : launch_sized<true, false>(g, pairs, op.act, stream);
  return fp8 ? launch_sized<false, true>(g, pairs, op.act, stream)
             : launch_sized<false, false>(g, pairs, op.act, stream);
}

}  // namespace moe
