// expert_forward.hip -- the experts' forward products over the packed rows:
//
//   gated block   z = x w_e^T + b_e (2F columns),  h = act(z[:F]) * z[F:]
//   linear layer  z = x w_e^T + b_e,               y = act(z) + residual
//
// Every sum is an fp32 MFMA accumulator; z, h and y are rounded once, to bf16,
// when they are stored (the activation sees the unrounded z).
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
//
// A workgroup takes tile after tile; the first loads of the next tile are issued before
// the results of the last leave, so that memory is not idle meanwhile.
template <class S, bool GLU, int ACT>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void forward_kernel(ForwardArgs g) {
  __shared__ __align__(1024) char smem[S::kLdsBytes];
  lds_ptr lds = (lds_ptr)smem;
  constexpr int kSize = S::FP8 ? 1 : 2;
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;  // columns of y in a tile
  constexpr int kWaveCols = kCols / S::WJ;        // and in a wave
  const int row_bytes = g.k * kSize, wrows = GLU ? 2 * g.n : g.n;
  const int steps = (row_bytes + S::SB - 1) / S::SB;
  const Wave<S> w = this_wave<S>();
  RowTiles<S::BI> order;
  order.init(g.offsets, g.counts, g.n_experts, g.rows, g.col_tiles);

  AlongLoader<S, S::LI> li;
  AlongLoader<S, S::LJ> lj;
  typename std::conditional<S::FP8, ScaleLoader, NoScales>::type sc;
  auto begin = [&](const RowTile &t) {
    const int j0 = t.j * kCols;
    li.init(static_cast<const char *>(g.x) + (static_cast<int64_t>(t.start) + t.i0) * row_bytes, row_bytes,
            [&](int r) {
              return r < S::BI && t.i0 + r < t.count ? static_cast<uint32_t>(r * row_bytes) : kNowhere;
            });
    lj.init(static_cast<const char *>(g.w) + static_cast<int64_t>(t.e) * wrows * row_bytes, row_bytes,
            [&](int r) {
              const int col = j0 + (GLU ? (r >> 5) * 16 + (r & 15) : r);
              const int row = GLU && (r & 16) ? g.n + col : col;
              return r < S::BJ && col < g.n ? static_cast<uint32_t>(row * row_bytes) : kNowhere;
            });
    if constexpr (S::FP8) {
      const int blocks = g.k / 128, tid = threadIdx.x;
      sc.rows = g.x_scales + (static_cast<int64_t>(t.start) + t.i0) * blocks;
      sc.row_off =
          tid < S::BI && t.i0 + tid < t.count ? static_cast<uint32_t>(tid * blocks * 4) : kNowhere;
      // the scales of a tile's weights: its gate and its up block, or its
      // 128-column blocks
      sc.weights = g.w_scales + static_cast<int64_t>(t.e) * (wrows / 128) * blocks;
      const int col = GLU ? j0 : j0 + tid * 128;
      const int block = (GLU && tid == 1 ? g.n + col : col) / 128;
      sc.weight_off = tid < (GLU ? 2 : (S::BJ + 127) / 128) && col < g.n
                          ? static_cast<uint32_t>(block * blocks * 4)
                          : kNowhere;
    }
    start<S>(lds, steps, li, lj, sc);
  };

  static_assert(S::WI * S::WJ * Transpose<kWaveCols>::kBytes <= S::kStage, "a region for each wave");
  auto scale_j = [&](int b) { return GLU ? b & 1 : (w.wj * S::FJ + b) * 16 / 128; };

  RowTile t = order.find(0);
  if (t.e < 0) return;
  begin(t);
  RowTile next;
  int younger = 0;  // stores after the tile's first loads
  auto one_tile = [&](auto blocks) {
    constexpr int FI = decltype(blocks)::value;
    f32x4 acc[FI][S::FJ];
    multiply<S, FI>(lds, steps, li, lj, sc, scale_j, younger, acc);
    // the last stage's LDS holds no load before multiply() begins: results pass
    // through it
    const int lane = late_lane_id();
    const Transpose<kWaveCols> turn{
        lds + (S::NST - 1) * S::kStage + wave_id() * Transpose<kWaveCols>::kBytes, lane};
    const float *bias = g.bias ? g.bias + static_cast<int64_t>(t.e) * wrows : nullptr;
    const int col0 = t.j * kCols + w.wj * kWaveCols;  // of the wave
    const int q4 = (lane >> 4) * 4, col = col0 + turn.col();
    const int left = t.count - t.i0;  // rows of the tile
    const int64_t row0 = static_cast<int64_t>(t.start) + t.i0;
    // read ahead of the next tile's loads, which would be waited for with them
    f32x4 shift[S::FJ];
#pragma unroll
    for (int b = 0; b < S::FJ; ++b) {
      const int c = col0 + (GLU ? b / 2 : b) * 16 + q4;
      shift[b] = bias && c < g.n ? *reinterpret_cast<const f32x4 *>(bias + (GLU && b % 2 ? g.n : 0) + c)
                                 : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    uint4 add[GLU ? 1 : FI][turn.kPasses];
    if constexpr (!GLU) {
      if (g.residual) {
        const auto residual = buffer_rsrc(g.residual + row0 * g.n, kRecords);
#pragma unroll
        for (int a = 0; a < FI; ++a)
#pragma unroll
          for (int p = 0; p < turn.kPasses; ++p) {
            const int i = (w.wi + a * S::WI) * 16 + turn.row(p);
            add[a][p] = __builtin_bit_cast(
                uint4, __builtin_amdgcn_raw_buffer_load_b128(
                           residual,
                           static_cast<int>(i < left && col < g.n ? (i * g.n + col) * 2u : kNowhere), 0,
                           kLoadDefault));
          }
      }
    }
    if (next.e >= 0) begin(next);

#pragma unroll
    for (int a = 0; a < FI; ++a) {
      const int i0 = (w.wi + a * S::WI) * 16;
      // what turn holds, to rows of `ld` columns from `to`
      auto leave = [&](uint16_t *to, int64_t ld, bool residual) {
        const auto r = buffer_rsrc(to + row0 * ld, kRecords);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int p = 0; p < turn.kPasses; ++p) {
          const int i = i0 + turn.row(p);
          float v[8];
          turn.get(p, v);
          if constexpr (!GLU) {
            if (residual) {
              float more[8];
              unpack8(add[a][p], more);
#pragma unroll
              for (int c = 0; c < 8; ++c) v[c] += more[c];
            }
          }
          store8(r, i < left && col < g.n ? static_cast<uint32_t>((i * ld + col) * 2) : kNowhere, v);
        }
        __builtin_amdgcn_wave_barrier();
      };
#pragma unroll
      for (int b = 0; b < S::FJ; ++b) acc[a][b] += shift[b];
      if (g.preact) {
        constexpr int kParts = GLU ? 2 : 1;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
#pragma unroll
          for (int b = part; b < S::FJ; b += kParts) turn.put(b / kParts, acc[a][b]);
          leave(g.preact + part * g.n, wrows, false);
        }
      }
#pragma unroll
      for (int b = 0; b < S::FJ; b += GLU ? 2 : 1) {
        f32x4 y;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          y[c] = act_value<ACT>(acc[a][b][c]) * (GLU ? acc[a][b + (GLU ? 1 : 0)][c] : 1.0f);
        turn.put(GLU ? b / 2 : b, y);
      }
      leave(g.y, g.n, g.residual != nullptr);
    }
    younger = FI * turn.kPasses;
  };
  for (int n = 1; t.e >= 0; ++n) {
    next = order.find(n);
    with_blocks<S>(t.count - t.i0, one_tile);
    t = next;
  }
}

template <class S, bool GLU>
hipError_t launch(ForwardArgs g, int64_t pairs, int act, hipStream_t stream) {
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;
  g.col_tiles = (g.n + kCols - 1) / kCols;
  const int64_t tiles = row_tile_bound<S::BI>(pairs, g.n_experts) * g.col_tiles;
  const uint32_t grid = tile_grid(tiles, S::kResident);
  return with_act(act, [&](auto a) {
    forward_kernel<S, GLU, decltype(a)::value><<<grid, S::kThreads, 0, stream>>>(g);
    return hipGetLastError();
  });
}

// Which tile: by the rows an expert has on average, and by whether larger tiles would
// leave compute units without work.
template <bool GLU, bool FP8>
hipError_t launch_sized(const ForwardArgs &g, int64_t pairs, int act, hipStream_t stream) {
  typedef Shape<16, 64, 1, 1, 128, 6, false, false, FP8> Few;
  typedef Shape<128, 128, 2, 2, 128, 2, false, false, FP8> Some;
  typedef Shape<256, 256, 2, 4, 128, 2, false, false, false> Many;
  const int64_t used = pairs < g.n_experts ? pairs : g.n_experts, rows = (pairs + used - 1) / used;
  const int64_t tiles = row_tile_bound<Some::BI>(pairs, g.n_experts) * ((g.n * (GLU ? 2 : 1) + 127) / 128);
  if (rows <= 16 && tiles < 4 * kComputeUnits) return launch<Few, GLU>(g, pairs, act, stream);
  if constexpr (!FP8) {
    if (rows > 112) return launch<Many, GLU>(g, pairs, act, stream);
  }
  return launch<Some, GLU>(g, pairs, act, stream);
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
