// expert_backward.hip -- gradients of the experts' products over the packed
// rows.  With dz the gradient at the product's result z = x w_e^T + b_e:
//
//   gated block   dz = (dh * up * act'(gate), dh * act(gate))
//   linear layer  dz = dy * act'(z)   (no activation: dz = dy)
//   dx = dz w_e     dw_e = dz^T x     dbias_e = sum over rows of dz
//
// dz is rounded to bf16 once, because both products read it through the bf16
// MFMA; dbias sums the unrounded values in fp32.
#include "expert_tile.hpp"

namespace moe {
namespace {

using namespace tile;

// ---- dz and the column sums ----------------------------------------------------

constexpr int kChunkRows = 64;   // rows of one workgroup (and of one partial sum)
constexpr int kSlabCols = 512;   // columns of a workgroup: 8 a lane
constexpr int kWaves = 4;

struct GradArgs {
  const uint16_t *dy, *preact;
  uint16_t *dz;
  float *partial;  // [chunks][width], or NULL
  const int32_t *offsets, *counts;
  int n_experts, rows, n, width, col_tiles;
};

__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4 *>(p), v);
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8]) {
  typedef __bf16 bf16x8s __attribute__((ext_vector_type(8)));
  bf16x8s r;
#pragma unroll
  for (int c = 0; c < 8; ++c) r[c] = static_cast<__bf16>(v[c]);
  *reinterpret_cast<bf16x8s *>(p) = r;
}

// One workgroup: up to 64 rows of one expert x 512 columns; a wave walks every
// fourth row.  Memory bound: each input is read and each output written once.
template <bool GLU, int ACT>
__global__ __launch_bounds__(kWaves *kWave) void grad_kernel(GradArgs g) {
  __shared__ float sums[kWaves][2][kSlabCols];
  const RowTile t = find_row_tile<kChunkRows>(g.offsets, g.counts, g.n_experts, g.rows, g.col_tiles);
  if (t.e < 0) return;
  const int wave = wave_id(), col = t.j * kSlabCols + lane_id() * 8;
  const bool live = col < g.n;
  float s0[8] = {}, s1[8] = {};
  const int end = min(t.count, t.i0 + kChunkRows);
  for (int i = t.i0 + wave; live && i < end; i += kWaves) {
    const int64_t row = static_cast<int64_t>(t.start) + i;
    float d[8], z[8];
    load8(g.dy + row * g.n + col, d);
    if constexpr (GLU) {
      float up[8];
      load8(g.preact + row * g.width + col, z);
      load8(g.preact + row * g.width + g.n + col, up);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float gate = z[c];
        z[c] = d[c] * act_value<ACT>(gate);
        d[c] = d[c] * up[c] * act_slope<ACT>(gate);
        s1[c] += z[c];
      }
      store8(g.dz + row * g.width + g.n + col, z);
    } else if constexpr (ACT != MOE_ACT_NONE) {
      load8(g.preact + row * g.n + col, z);
#pragma unroll
      for (int c = 0; c < 8; ++c) d[c] *= act_slope<ACT>(z[c]);
    }
    if (GLU || ACT != MOE_ACT_NONE) store8(g.dz + row * g.width + col, d);
#pragma unroll
    for (int c = 0; c < 8; ++c) s0[c] += d[c];
  }
  if (!g.partial) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    sums[wave][0][lane_id() * 8 + c] = s0[c];
    if (GLU) sums[wave][1][lane_id() * 8 + c] = s1[c];
  }
  __syncthreads();
  // chunk number: chunks of the experts before, then this one's
  const int64_t chunk = t.start / kChunkRows + t.e + t.i0 / kChunkRows;
  for (int c = threadIdx.x; c < kSlabCols; c += kWaves * kWave) {
    const int at = t.j * kSlabCols + c;
    if (at >= g.n) break;
#pragma unroll
    for (int h = 0; h < (GLU ? 2 : 1); ++h) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += sums[w][h][c];
      g.partial[chunk * g.width + h * g.n + at] = v;
    }
  }
}

// dbias[e][c]: the expert's partial sums in row order.
__global__ __launch_bounds__(256) void bias_kernel(GradArgs g, float *dbias) {
  const int e = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= g.width) return;
  const ExpertRows r = expert_rows(g.offsets, g.counts, e, g.rows);
  const int64_t first = r.start / kChunkRows + e;
  double v = 0.0;
  for (int q = 0; q < (r.count + kChunkRows - 1) / kChunkRows; ++q) v += g.partial[(first + q) * g.width + c];
  dbias[static_cast<int64_t>(e) * g.width + c] = static_cast<float>(v);
}

template <bool GLU>
hipError_t launch_grad(GradArgs g, int64_t pairs, int act, hipStream_t stream) {
  g.col_tiles = (g.n + kSlabCols - 1) / kSlabCols;
  const int64_t tiles = row_tile_bound<kChunkRows>(pairs, g.n_experts) * g.col_tiles;
  if (tiles == 0) return hipSuccess;
  return with_act(act, [&](auto a) {
    grad_kernel<GLU, decltype(a)::value>
        <<<static_cast<uint32_t>((tiles + 7) / 8 * 8), kWaves * kWave, 0, stream>>>(g);
    return hipGetLastError();
  });
}

// ---- dx = dz w -------------------------------------------------------------------

struct ProductArgs {
  const uint16_t *dz, *x, *w;
  uint16_t *out;
  const int32_t *offsets, *counts;
  int n_experts, rows;
  int k, n;       // columns of x and of dz
  int col_tiles;
};

__device__ __forceinline__ bf16x4 to_bf16(const f32x4 v) {
  bf16x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = static_cast<__bf16>(v[i]);
  return r;
}

template <class S>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void dx_kernel(ProductArgs g) {
  __shared__ __align__(1024) char smem[S::kLdsBytes];
  const RowTile t = find_row_tile<S::BI>(g.offsets, g.counts, g.n_experts, g.rows, g.col_tiles);
  if (t.e < 0) return;
  const int row_bytes = g.n * 2, j0 = t.j * S::BJ;
  const int wave = wave_id(), wi = wave / S::WJ, wj = wave % S::WJ, lane = lane_id();
  AlongLoader<S, S::LI> li;
  li.init(g.dz + (static_cast<int64_t>(t.start) + t.i0) * g.n, row_bytes, [&](int r) {
    return r < S::BI && t.i0 + r < t.count ? static_cast<uint32_t>(r * row_bytes) : kNowhere;
  });
  AcrossLoader<S, S::BJ, S::LJ> lj;
  lj.init(g.w + static_cast<int64_t>(t.e) * g.n * g.k + j0, static_cast<int64_t>(g.k) * 2, g.n, g.k - j0);
  f32x4 acc[S::FI][S::FJ];
  multiply<S>((lds_ptr)smem, (g.n + kStepRows - 1) / kStepRows, li, lj, NoScales(), [](int) { return 0; },
              wi, wj, acc);
#pragma unroll
  for (int b = 0; b < S::FJ; ++b) {
    const int col = j0 + (wj * S::FJ + b) * 16 + (lane >> 4) * 4;
    if (col >= g.k) continue;
#pragma unroll
    for (int a = 0; a < S::FI; ++a) {
      const int i = t.i0 + (wi * S::FI + a) * 16 + (lane & 15);
      if (i < t.count)
        *reinterpret_cast<bf16x4 *>(g.out + (static_cast<int64_t>(t.start) + i) * g.k + col) =
            to_bf16(acc[a][b]);
    }
  }
}

// ---- dw = dz^T x -----------------------------------------------------------------

// One workgroup a BI x BJ tile of one expert's dw: the contraction runs over
// the expert's rows, none of them for an expert without rows (its dw is zeros).
template <class S>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void dw_kernel(ProductArgs g, int row_tiles, int total) {
  __shared__ __align__(1024) char smem[S::kLdsBytes];
  // an XCD takes one run of tiles, expert by expert: its rows stay in that L2
  const int chunk = (total + 7) / 8, pos = blockIdx.x / 8;
  const int64_t id = static_cast<int64_t>(blockIdx.x % 8) * chunk + pos;
  if (pos >= chunk || id >= total) return;
  const int per = row_tiles * g.col_tiles;
  const int e = static_cast<int>(id / per), q = static_cast<int>(id - static_cast<int64_t>(e) * per);
  const int group = q / (8 * g.col_tiles), rest = q - group * 8 * g.col_tiles;
  const int size = min(8, row_tiles - group * 8);
  const int j0 = rest / size * S::BJ, i0 = (group * 8 + rest % size) * S::BI;
  const ExpertRows r = expert_rows(g.offsets, g.counts, e, g.rows);
  const int wave = wave_id(), wi = wave / S::WJ, wj = wave % S::WJ, lane = lane_id();
  AcrossLoader<S, S::BI, S::LI> li;
  li.init(g.dz + static_cast<int64_t>(r.start) * g.n + i0, static_cast<int64_t>(g.n) * 2, r.count, g.n - i0);
  AcrossLoader<S, S::BJ, S::LJ> lj;
  lj.init(g.x + static_cast<int64_t>(r.start) * g.k + j0, static_cast<int64_t>(g.k) * 2, r.count, g.k - j0);
  f32x4 acc[S::FI][S::FJ];
  multiply<S>((lds_ptr)smem, (r.count + kStepRows - 1) / kStepRows, li, lj, NoScales(),
              [](int) { return 0; }, wi, wj, acc);
  uint16_t *out = g.out + static_cast<int64_t>(e) * g.n * g.k;
#pragma unroll
  for (int b = 0; b < S::FJ; ++b) {
    const int col = j0 + (wj * S::FJ + b) * 16 + (lane >> 4) * 4;
    if (col >= g.k) continue;
#pragma unroll
    for (int a = 0; a < S::FI; ++a) {
      const int i = i0 + (wi * S::FI + a) * 16 + (lane & 15);
      if (i < g.n) *reinterpret_cast<bf16x4 *>(out + static_cast<int64_t>(i) * g.k + col) = to_bf16(acc[a][b]);
    }
  }
}

template <class S>
hipError_t launch_dx(ProductArgs g, int64_t pairs, hipStream_t stream) {
  g.col_tiles = (g.k + S::BJ - 1) / S::BJ;
  const int64_t tiles = row_tile_bound<S::BI>(pairs, g.n_experts) * g.col_tiles;
  if (tiles == 0) return hipSuccess;
  dx_kernel<S><<<static_cast<uint32_t>((tiles + 7) / 8 * 8), S::kThreads, 0, stream>>>(g);
  return hipGetLastError();
}

template <class S>
hipError_t launch_dw(ProductArgs g, hipStream_t stream) {
  g.col_tiles = (g.k + S::BJ - 1) / S::BJ;
  const int row_tiles = (g.n + S::BI - 1) / S::BI;
  const int64_t total = static_cast<int64_t>(g.n_experts) * row_tiles * g.col_tiles;
  dw_kernel<S><<<static_cast<uint32_t>((total + 7) / 8 * 8), S::kThreads, 0, stream>>>(
      g, row_tiles, static_cast<int>(total));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_backward(const moe_problem &p, const moe_plan &plan, const moe_expert_op &op,
                                  bool glu, const ExpertBackward &b, hipStream_t stream) {
  const int64_t pairs = expert_row_bound(p);
  const int width = glu ? 2 * op.out_dim : op.out_dim;
  const bool through_act = glu || op.act != MOE_ACT_NONE;
  hipError_t err = hipSuccess;
  if (through_act || b.dbias) {
    GradArgs g;
    g.dy = b.dy;
    g.preact = b.preact;
    g.dz = b.dz;
    g.partial = b.dbias ? static_cast<float *>(b.workspace) : nullptr;
    g.offsets = plan.expert_offsets;
    g.counts = plan.expert_counts;
    g.n_experts = p.n_experts;
    g.rows = static_cast<int>(max_rows(p));
    g.n = op.out_dim;
    g.width = width;
    err = glu ? launch_grad<true>(g, pairs, op.act, stream) : launch_grad<false>(g, pairs, op.act, stream);
    if (err != hipSuccess) return err;
    if (b.dbias) {
      bias_kernel<<<dim3((width + 255) / 256, p.n_experts), 256, 0, stream>>>(g, b.dbias);
      err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
  }
  ProductArgs a;
  a.dz = through_act ? b.dz : b.dy;
  a.x = b.x;
  a.w = b.w;
  a.offsets = plan.expert_offsets;
  a.counts = plan.expert_counts;
  a.n_experts = p.n_experts;
  a.rows = static_cast<int>(max_rows(p));
  a.k = op.in_dim;
  a.n = width;
  if (b.dx) {
    a.out = b.dx;
    err = launch_dx<Shape<128, 128, 2, 2, 2, false, true>>(a, pairs, stream);
    if (err != hipSuccess) return err;
  }
  if (b.dw) {
    a.out = b.dw;
    err = launch_dw<Shape<128, 128, 2, 2, 2, true, true>>(a, stream);
  }
  return err;
}

}  // namespace moe
