// expert_mx.hip -- the experts' products with MX-FP4 weights over the packed rows (MX-FP4 or
// FP8):
//
//   gated block   z = x w_e^T + b_e (2F columns),  h = act(z[:F]) * z[F:]
//   linear layer  z = x w_e^T + b_e,               y = act(z) + residual
//
// Sums are fp32 accumulators of the scaled matrix instruction (mx_tile.hpp says what it keeps
// of its terms).  h and y are rounded once: to bf16, or h to MX-FP4 with the scale of
// its own 32 values, the rows of the next product.
#include "expert_tile.hpp"
#include "mx_encode.hpp"
#include "mx_tile.hpp"

namespace moe {
namespace {

using namespace tile;

struct MxArgs {
  const char *x, *x_scales, *w, *w_scales;
  const float *bias;
  const uint16_t *residual;
  uint16_t *y;
  uint8_t *codes, *scales;  // instead of y
  const int32_t *offsets, *counts;
  int n_experts, rows;
  int k, n;  // columns of a row of x; columns of y
  int act;
  int col_tiles;
};

// GLU: 16-row blocks of gate and up rows in turn (as the other formats' products).
struct MxGateUpRow {
  int n;
  __device__ __forceinline__ uint32_t operator()(int r) const {
    return (r & 16 ? n : 0) + (r >> 5) * 16 + (r & 15);
  }
};

__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case MOE_ACT_SILU: return act_value<MOE_ACT_SILU>(z);
    case MOE_ACT_GELU_TANH: return act_value<MOE_ACT_GELU_TANH>(z);
    case MOE_ACT_RELU: return act_value<MOE_ACT_RELU>(z);
    default: return z;
  }
}

// As with_blocks; a tile of six blocks a wave goes by single ones.
template <class S, class F>
__device__ __forceinline__ void with_own_blocks(int rows, F f) {
  if constexpr (S::FI == 6) {
    const int blocks = (rows + 16 * S::WI - 1) / (16 * S::WI);
    if (blocks <= 2) return f(std::integral_constant<int, 2>());
    if (blocks == 3) return f(std::integral_constant<int, 3>());
    if (blocks == 4) return f(std::integral_constant<int, 4>());
    if (blocks == 5) return f(std::integral_constant<int, 5>());
    return f(std::integral_constant<int, 6>());
  } else {
    with_blocks<S>(rows, f);
  }
}

template <class S, bool GLU>
__global__ __launch_bounds__(S::kThreads *S::WK, S::kWavesPerSimd) void mx_kernel(MxArgs g) {
  __shared__ __align__(1024) char smem[S::kLdsBytes];
  lds_ptr lds = (lds_ptr)smem + group_id<S>() * S::kGroupLds;
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;  // columns of y in a tile
  constexpr int kWaveCols = kCols / S::WJ;        // and in a wave
  const int x_bytes = S::FP8 ? g.k : g.k / 2, w_bytes = g.k / 2, blocks = g.k / 32;
  const int x_scale_bytes = S::FP8 ? g.k / 128 * 4 : blocks;
  const int wrows = GLU ? 2 * g.n : g.n;
  const Wave<S> w = this_wave<S>();
  RowTiles<S::BI> order;
  order.init(g.offsets, g.counts, g.n_experts, g.rows, g.col_tiles);
  RowTile t = order.find(0);
  if (t.e < 0) return;

  typedef typename std::conditional<GLU, MxGateUpRow, SameRow>::type WeightRow;
  MxFeed<S, WeightRow> feed;
  if constexpr (GLU) feed.j.row.n = feed.w.row.n = g.n;
  feed.i.init(x_bytes);
  feed.j.init(w_bytes);
  feed.x.init(x_scale_bytes);
  feed.w.init(blocks);
  auto source = [&](const RowTile &r) {
    if (r.e < 0) return kNoMxSource;
    const int j0 = r.j * kCols, left = min(r.count - r.i0, S::BI);
    const int64_t row0 = static_cast<int64_t>(r.start) + r.i0, wrow0 = static_cast<int64_t>(r.e) * wrows + j0;
    MxSource s = kNoMxSource;
    s.i = {g.x + row0 * x_bytes, left * x_bytes, 0};
    s.j = {g.w + wrow0 * w_bytes, (wrows - j0) * w_bytes, 0};
    s.x = {g.x_scales + row0 * x_scale_bytes, left * x_scale_bytes};
    s.w = {g.w_scales + wrow0 * blocks, (wrows - j0) * blocks};
    // of a group
    s.steps = (w_bytes + kStepBytes * S::kSpan * S::WK - 1) / (kStepBytes * S::kSpan * S::WK) * S::kSpan;
    if constexpr (S::WK == 1) s.steps = (w_bytes + kStepBytes - 1) / kStepBytes;
    return s;
  };

  MxSource cur = source(t), following;
  MxProgress at;
  start_mx<S>(lds, feed, cur, at);
  auto one_tile = [&](auto own_blocks) {
    constexpr int FI = decltype(own_blocks)::value;
    constexpr int kTurnCols = GLU ? kWaveCols : S::kTurnCols, kTurns = kWaveCols / kTurnCols;
    constexpr int kTurnBlocks = kTurnCols / 16;
    f32x4 acc[FI][S::FJ];
    multiply_mx<S, FI>(lds, feed, cur, following, blocks, at, acc);
    const int lane = late_lane_id();
    if constexpr (S::WK > 1) {
      // the groups' sums, added in order by the first, through what is its way out
      lds_ptr sums = lds + S::kLoadLds + lane * 16;
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
    const Transpose<kTurnCols> turn{lds + S::kLoadLds + group_wave<S>() * Transpose<kTurnCols>::kBytes, lane};
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
    // where pass p of block row a goes: row and column of its eight values; past the
    // results' end kNowhere
    auto row_of = [&](int a, int p) { return (w.wi + a * S::WI) * 16 + turn.row(p); };
    auto place = [&](int a, int p, int h) {
      const int i = row_of(a, p), col = col0 + h * kTurnCols + turn.col();
      return i < left && col < g.n ? static_cast<uint32_t>(i * g.n + col) : kNowhere;
    };
    auto in_bytes = [](uint32_t at, int shift_left) { return at == kNowhere ? kNowhere : at << shift_left; };
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
                  uint4, __builtin_amdgcn_raw_buffer_load_b128(
                             r, static_cast<int>(in_bytes(place(a, p, h), 1)), 0, kLoadDefault));
      }
    }
#pragma unroll
    for (int a = 0; a < FI; ++a) {
#pragma unroll
      for (int b = 0; b < S::FJ; ++b) acc[a][b] += shift[b];
#pragma unroll
      for (int h = 0; h < kTurns; ++h) {
#pragma unroll
        for (int b = 0; b < kTurnBlocks; ++b) {
          const int at_b = (h * kTurnBlocks + b) * (GLU ? 2 : 1);
          f32x4 y;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            y[c] = activate(g.act, acc[a][at_b][c]) * (GLU ? acc[a][at_b + (GLU ? 1 : 0)][c] : 1.0f);
          turn.put(b, y);
        }
        __builtin_amdgcn_wave_barrier();
        if (GLU && g.codes) {
          const auto rc = buffer_rsrc(g.codes + row0 * (g.n / 2), kRecords);
          const auto rs = buffer_rsrc(g.scales + row0 * (g.n / 32), kRecords);
#pragma unroll
          for (int p = 0; p < turn.kPasses; ++p) {
            float v[8];
            turn.get(p, v);
            uint32_t scale;
            const uint32_t c = mx_encode8(v, scale);  // (n is a multiple of 32: whole blocks are in or out)
            const uint32_t to = place(a, p, h);
            __builtin_amdgcn_raw_buffer_store_b32(c, rc, static_cast<int>(to == kNowhere ? to : to / 2), 0, 0);
            const bool leads = to != kNowhere && (lane & 3) == 0;
            __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(scale), rs,
                                                 static_cast<int>(leads ? to / 32 : kNowhere), 0, 0);
          }
        } else {
          const auto r = buffer_rsrc(g.y + row0 * g.n, kRecords);
#pragma unroll
          for (int p = 0; p < turn.kPasses; ++p) {
            float v[8];
            turn.get(p, v);
            if constexpr (!GLU) {
              if (g.residual) {
                float more[8];
                unpack8(add[a][h][p], more);
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] += more[c];
              }
            }
            store8(r, in_bytes(place(a, p, h), 1), v);
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
    at.younger = FI * kTurns * turn.kPasses;
  };
  for (int n = 1; t.e >= 0; ++n) {
    const RowTile next = order.find(n);
    following = source(next);
    with_own_blocks<S>(t.count - t.i0, one_tile);
    t = next;
    cur = following;
  }
  wait_and_meet<0>();  // loads past the last tile fetch nothing, but write LDS
}

// resident: tile_grid's
template <class S, bool GLU>
hipError_t launch(MxArgs g, int64_t pairs, hipStream_t stream, int resident = S::kResident) {
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;
  g.col_tiles = (g.n + kCols - 1) / kCols;
  const int64_t tiles = row_tile_bound<S::BI>(pairs, g.n_experts) * g.col_tiles;
  mx_kernel<S, GLU><<<tile_grid(tiles, resident), S::kThreads * S::WK, 0, stream>>>(g);
  return hipGetLastError();
}

template <bool GLU, bool FP8, bool ODD>
hipError_t launch_sized(const MxArgs &g, int64_t pairs, hipStream_t stream) {
  typedef MxShape<16, 64, 1, 1, FP8 ? 2 : 3, FP8, ODD, 4> Split;
  typedef MxShape<16, 64, 1, 1, 4, FP8, ODD> Few;
  typedef MxShape<64, 128, 2, 2, 3, FP8, ODD> Low;
  typedef MxShape<128, 128, 2, 2, 2, FP8, ODD> Some;
  typedef typename std::conditional<FP8, MxShape<128, 256, 2, 4, 2, FP8, ODD>,
                                    MxShape<256, 256, 2, 4, 2, FP8, ODD>>::type Many;
  typedef MxShape<FP8 ? 128 : 384, FP8 ? 256 : 128, FP8 ? 2 : 4, FP8 ? 4 : 2, 2, FP8, ODD> Tall;
  const int64_t used = pairs < g.n_experts ? pairs : g.n_experts, rows = (pairs + used - 1) / used;
  const int wrows = g.n * (GLU ? 2 : 1);
  const int64_t tiles = row_tile_bound<Some::BI>(pairs, g.n_experts) * col_tiles<Some::BJ>(wrows);
  const int64_t split_tiles = row_tile_bound<Split::BI>(pairs, g.n_experts) * col_tiles<Split::BJ>(wrows);
  if (g.k >= 2048 && (rows <= 12 || split_tiles <= 2 * kComputeUnits)) return launch<Split, GLU>(g, pairs, stream);
  if (rows <= 16 && tiles < 4 * kComputeUnits) return launch<Few, GLU>(g, pairs, stream);
  if (tiles < kEnoughTiles) return launch<Low, GLU>(g, pairs, stream);
  if (rows <= 112) return launch<Some, GLU>(g, pairs, stream);
  if (!FP8 && rows < 336) return launch<Tall, GLU>(g, pairs, stream);
  if (row_tile_bound<Many::BI>(pairs, g.n_experts) * col_tiles<Many::BJ>(wrows) < kEnoughTiles)
    return launch<Some, GLU>(g, pairs, stream);
  return launch<Many, GLU>(g, pairs, stream);
}

template <bool GLU>
hipError_t launch_format(const MxArgs &g, bool fp8, int64_t pairs, hipStream_t stream) {
  if (fp8) return launch_sized<GLU, true, false>(g, pairs, stream);
  return g.k % 128 ? launch_sized<GLU, false, true>(g, pairs, stream)
                   : launch_sized<GLU, false, false>(g, pairs, stream);
}

}  // namespace

hipError_t launch_expert_mx(const moe_problem &p, const moe_plan &plan, const moe_expert_op &op, bool glu,
                            const ExpertMx &f, hipStream_t stream) {
  const int64_t rows = max_rows(p), pairs = expert_row_bound(p);
  if (pairs == 0) return hipSuccess;
  MxArgs g;
  g.x = static_cast<const char *>(f.x);
  g.x_scales = static_cast<const char *>(f.x_scales);
  g.w = reinterpret_cast<const char *>(f.w);
  g.w_scales = reinterpret_cast<const char *>(f.w_scales);
  g.bias = f.bias;
  g.residual = f.residual;
  g.y = f.y_scales ? nullptr : static_cast<uint16_t *>(f.y);
  g.codes = f.y_scales ? static_cast<uint8_t *>(f.y) : nullptr;
  g.scales = f.y_scales;
  g.offsets = plan.expert_offsets;
  g.counts = plan.expert_counts;
  g.n_experts = p.n_experts;
  g.rows = static_cast<int>(rows);
  g.k = op.in_dim;
  g.n = op.out_dim;
  g.act = op.act;
  const bool fp8 = op.fmt == MOE_FMT_FP8_E4M3_B128;
  return glu ? launch_format<true>(g, fp8, pairs, stream) : launch_format<false>(g, fp8, pairs, stream);
}

}  // namespace moe
