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

__device__ __forceinline__ bf16x4 to_bf16(const f32x4 v) {
  bf16x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = static_cast<__bf16>(v[i]);
  return r;
}

// GLU: a tile holds BJ / 2 columns of h; its weight rows go to LDS as
// alternating 16-row blocks of gate and up rows, so that a wave holds both
// halves of each of its columns and the product is formed in registers.
template <class S, bool GLU, int ACT>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void forward_kernel(ForwardArgs g) {
  __shared__ __align__(1024) char smem[S::kLdsBytes];
  const RowTile t = find_row_tile<S::BI>(g.offsets, g.counts, g.n_experts, g.rows, g.col_tiles);
  if (t.e < 0) return;
  constexpr int kSize = S::FP8 ? 1 : 2;
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;  // columns of y in a tile
  const int row_bytes = g.k * kSize, wrows = GLU ? 2 * g.n : g.n;
  const int j0 = t.j * kCols;
  const int wave = wave_id(), wi = wave / S::WJ, wj = wave % S::WJ, lane = lane_id();

  AlongLoader<S, S::LI> li;
  li.init(static_cast<const char *>(g.x) + (static_cast<int64_t>(t.start) + t.i0) * row_bytes, row_bytes,
          [&](int r) {
            return r < S::BI && t.i0 + r < t.count ? static_cast<uint32_t>(r * row_bytes) : kNowhere;
          });
  AlongLoader<S, S::LJ> lj;
  lj.init(static_cast<const char *>(g.w) + static_cast<int64_t>(t.e) * wrows * row_bytes, row_bytes,
          [&](int r) {
            const int col = j0 + (GLU ? (r >> 5) * 16 + (r & 15) : r);
            const int row = GLU && (r & 16) ? g.n + col : col;
            return r < S::BJ && col < g.n ? static_cast<uint32_t>(row * row_bytes) : kNowhere;
          });
  f32x4 acc[S::FI][S::FJ];
  const int steps = (row_bytes + kStepBytes - 1) / kStepBytes;
  lds_ptr lds = (lds_ptr)smem;
  if constexpr (S::FP8) {
    const int blocks = g.k / 128, tid = threadIdx.x;
    ScaleLoader sc;
    sc.rows = g.x_scales + (static_cast<int64_t>(t.start) + t.i0) * blocks;
    sc.row_off = tid < S::BI && t.i0 + tid < t.count ? static_cast<uint32_t>(tid * blocks * 4) : kNowhere;
    // the scales of a tile's weights: its gate and its up block, or its
    // 128-column blocks
    sc.weights = g.w_scales + static_cast<int64_t>(t.e) * (wrows / 128) * blocks;
    const int col = GLU ? j0 : j0 + tid * 128;
    const int block = (GLU && tid == 1 ? g.n + col : col) / 128;
    sc.weight_off = tid < (GLU ? 2 : (S::BJ + 127) / 128) && col < g.n
                        ? static_cast<uint32_t>(block * blocks * 4)
                        : kNowhere;
    multiply<S>(lds, steps, li, lj, sc,
                [&](int b) { return GLU ? b & 1 : (wj * S::FJ + b) * 16 / 128; }, wi, wj, acc);
  } else {
    multiply<S>(lds, steps, li, lj, NoScales(), [](int) { return 0; }, wi, wj, acc);
  }

  const float *bias = g.bias ? g.bias + static_cast<int64_t>(t.e) * wrows : nullptr;
  const int q4 = (lane >> 4) * 4;
#pragma unroll
  for (int b = 0; b < S::FJ; b += GLU ? 2 : 1) {
    const int col = j0 + (GLU ? (wj * S::FJ + b) * 8 : (wj * S::FJ + b) * 16) + q4;
    if (col >= g.n) continue;
    f32x4 b0{0.f, 0.f, 0.f, 0.f}, b1 = b0;
    if (bias) {
      b0 = *reinterpret_cast<const f32x4 *>(bias + col);
      if (GLU) b1 = *reinterpret_cast<const f32x4 *>(bias + g.n + col);
    }
#pragma unroll
    for (int a = 0; a < S::FI; ++a) {
      const int i = t.i0 + (wi * S::FI + a) * 16 + (lane & 15);
      if (i >= t.count) continue;
      const int64_t row = static_cast<int64_t>(t.start) + i;
      const f32x4 z = acc[a][b] + b0;
      f32x4 y;
      if constexpr (GLU) {
        const f32x4 up = acc[a][b + 1] + b1;
        if (g.preact) {
          *reinterpret_cast<bf16x4 *>(g.preact + row * wrows + col) = to_bf16(z);
          *reinterpret_cast<bf16x4 *>(g.preact + row * wrows + g.n + col) = to_bf16(up);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = act_value<ACT>(z[c]) * up[c];
      } else {
        if (g.preact) *reinterpret_cast<bf16x4 *>(g.preact + row * wrows + col) = to_bf16(z);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = act_value<ACT>(z[c]);
        if (g.residual) {
          const bf16x4 r = *reinterpret_cast<const bf16x4 *>(g.residual + row * g.n + col);
#pragma unroll
          for (int c = 0; c < 4; ++c) y[c] += static_cast<float>(r[c]);
        }
      }
      *reinterpret_cast<bf16x4 *>(g.y + row * g.n + col) = to_bf16(y);
    }
  }
}

template <class S, bool GLU>
hipError_t launch(ForwardArgs g, int64_t pairs, int act, hipStream_t stream) {
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;
  g.col_tiles = (g.n + kCols - 1) / kCols;
  const int64_t tiles = row_tile_bound<S::BI>(pairs, g.n_experts) * g.col_tiles;
  const dim3 grid(static_cast<uint32_t>((tiles + 7) / 8 * 8));
  return with_act(act, [&](auto a) {
    forward_kernel<S, GLU, decltype(a)::value><<<grid, S::kThreads, 0, stream>>>(g);
    return hipGetLastError();
  });
}

template <bool GLU, bool FP8>
hipError_t launch_sized(const ForwardArgs &g, int64_t pairs, int act, hipStream_t stream) {
  return launch<Shape<128, 128, 2, 2, 2, false, false, FP8>, GLU>(g, pairs, act, stream);
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
