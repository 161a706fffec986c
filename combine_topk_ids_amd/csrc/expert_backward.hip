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

// Rows of one workgroup (and of one partial sum): one batch of its waves.  (64
// rows: 15.1 us against 7.2 at 999 rows of 2 x 712 columns, 70.2 against 66.8 at 24576
// of 2 x 1024.)
constexpr int kChunkRows = kBiasChunkRows;
constexpr int kSlabCols = kGradCols;  // columns of a workgroup: 8 a lane
constexpr int kWaves = 4;
constexpr int kBatch = 4;

struct GradArgs {
  const uint16_t *dy, *preact;
  uint16_t *dz;
  float *partial;  // [chunks][width], or NULL
  const int32_t *offsets, *counts;
  int n_experts, rows, n, width, col_tiles;
};

// One workgroup: up to 16 rows of one expert x 512 columns; a wave takes every
// fourth row.  Memory bound: each input is read and each output written once.
template <bool GLU, int ACT>
__global__ __launch_bounds__(kWaves *kWave) void grad_kernel(GradArgs g) {
  __shared__ float sums[kWaves][2][kSlabCols];
  RowTiles<kChunkRows> order;
  order.init(g.offsets, g.counts, g.n_experts, g.rows, g.col_tiles);
  const RowTile t = order.find(0);
  if (t.e < 0) return;
  const int wave = wave_id(), col = t.j * kSlabCols + lane_id() * 8;
  const bool live = col < g.n;
  float s0[8] = {}, s1[8] = {};
  const int end = min(t.count, t.i0 + kChunkRows);
  static_assert(kChunkRows == kWaves * kBatch, "one batch a wave: its loads are in flight together");
  const int i = t.i0 + wave;
  if (live && i < end) {
    uint4 rd[kBatch], rz[kBatch], ru[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t row = static_cast<int64_t>(t.start) + min(i + u * kWaves, end - 1);
      rd[u] = *reinterpret_cast<const uint4 *>(g.dy + row * g.n + col);
      if (GLU || ACT != MOE_ACT_NONE) rz[u] = *reinterpret_cast<const uint4 *>(g.preact + row * g.width + col);
      if (GLU) ru[u] = *reinterpret_cast<const uint4 *>(g.preact + row * g.width + g.n + col);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (i + u * kWaves >= end) break;
      const int64_t row = static_cast<int64_t>(t.start) + i + u * kWaves;
      float d[8], z[8];
      unpack8(rd[u], d);
      if constexpr (GLU) {
        float up[8];
        unpack8(rz[u], z);
        unpack8(ru[u], up);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float gate = z[c];
          z[c] = d[c] * act_value<ACT>(gate);
          d[c] = d[c] * up[c] * act_slope<ACT>(gate);
          s1[c] += z[c];
        }
        store8(g.dz + row * g.width + g.n + col, z);
      } else if constexpr (ACT != MOE_ACT_NONE) {
        unpack8(rz[u], z);
#pragma unroll
        for (int c = 0; c < 8; ++c) d[c] *= act_slope<ACT>(z[c]);
      }
      if (GLU || ACT != MOE_ACT_NONE) store8(g.dz + row * g.width + col, d);
#pragma unroll
      for (int c = 0; c < 8; ++c) s0[c] += d[c];
    }
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

// dbias[e][c]: the expert's partial sums, 16 columns a workgroup.  Thread (q, c) adds
// every 16th chunk's; then the 16 are added in order.  (One thread a column took 148 us
// for 7876 rows: a chain of 492 loads.)
__global__ __launch_bounds__(256) void bias_kernel(GradArgs g, float *dbias) {
  __shared__ double sums[16][16];
  const int e = blockIdx.y, c = threadIdx.x % 16, q0 = threadIdx.x / 16, col = blockIdx.x * 16 + c;
  const ExpertRows r = expert_rows(g.offsets, g.counts, e, g.rows);
  const float *from = g.partial + (r.start / kChunkRows + static_cast<int64_t>(e)) * g.width + col;
  const int chunks = (r.count + kChunkRows - 1) / kChunkRows;
  double v = 0.0;
  if (col < g.width) {
#pragma unroll 4
    for (int q = q0; q < chunks; q += 16) v += from[static_cast<int64_t>(q) * g.width];
  }
  sums[q0][c] = v;
  __syncthreads();
  if (q0 != 0 || col >= g.width) return;
#pragma unroll
  for (int q = 1; q < 16; ++q) v += sums[q][c];
  dbias[static_cast<int64_t>(e) * g.width + col] = static_cast<float>(v);
}

template <bool GLU>
hipError_t launch_grad(GradArgs g, int64_t groups, int act, hipStream_t stream) {
  static_assert(kSlabCols == 8 * kWave && kWaves * kWave == kGradThreads, "the launch that the checks bound");
  g.col_tiles = (g.n + kSlabCols - 1) / kSlabCols;
  if (groups == 0) return hipSuccess;
  return with_act(act, [&](auto a) {
    grad_kernel<GLU, decltype(a)::value>
        <<<static_cast<uint32_t>(groups), kWaves * kWave, 0, stream>>>(g);
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
  float *parts;   // dw's, where its rows are split
};

// Results of a wave, to a tile of rows x cols of `out`, whose rows have `ld`
// columns.  Returns the wave's stores.
// T: uint16_t (bf16, rounded here) or float.  POLICY: cache bits of the bf16 stores.
template <class S, int FI, int POLICY, class T>
__device__ __forceinline__ int store_tile(lds_ptr lds, const f32x4 (&acc)[FI][S::FJ], T *out, int ld, int rows,
                                          int cols) {
  constexpr int kSize = sizeof(T);
  const Wave<S> w = this_wave<S>();
  const auto turn = Transpose<S::kWaveCols>::template make<S>(lds, late_lane_id());
  const int col = w.wj * S::kWaveCols + turn.col();
  const auto r = buffer_rsrc(out, kRecords);
#pragma unroll
  for (int a = 0; a < FI; ++a) {
#pragma unroll
    for (int b = 0; b < S::FJ; ++b) turn.put(b, acc[a][b]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < turn.kPasses; ++p) {
      const int i = (w.wi + a * S::WI) * 16 + turn.row(p);
      float v[8];
      turn.get(p, v);
      const uint32_t at = i < rows && col < cols ? static_cast<uint32_t>(i * ld + col) * kSize : kNowhere;
      if constexpr (kSize == 2)
        store8<POLICY>(r, at, v);
      else
        store8_f32(r, at, v);
    }
    __builtin_amdgcn_wave_barrier();
  }
  return FI * turn.kPasses * (kSize / 2);
}

template <class S>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void dx_kernel(ProductArgs g) {
  __shared__ __align__(1024) char smem[S::kLdsBytes];
  lds_ptr lds = (lds_ptr)smem;
  RowTiles<S::BI> order;
  order.init(g.offsets, g.counts, g.n_experts, g.rows, g.col_tiles);
  RowTile t = order.find(0);
  if (t.e < 0) return;
  Feed<S, Along<S, S::LI, SameRow>, Across<S, S::BJ, S::LJ>, NoScaleLanes> feed;
  feed.i.init(g.n * 2);
  feed.j.init(g.k * 2);
  auto source = [&](const RowTile &r) {
    Source s = kNoSource;
    if (r.e < 0) return s;
    const int j0 = r.j * S::BJ;
    s.i = {reinterpret_cast<const char *>(g.dz + (static_cast<int64_t>(r.start) + r.i0) * g.n),
           min(r.count - r.i0, S::BI) * g.n * 2, 0};
    s.j = {reinterpret_cast<const char *>(g.w + static_cast<int64_t>(r.e) * g.n * g.k + j0), g.n, j0 * 2};
    s.steps = (g.n + kStepRows - 1) / kStepRows;
    return s;
  };
  Source cur = source(t), following;
  start<S>(lds, feed, cur);
  Progress at;
  auto one_tile = [&](auto blocks) {
    constexpr int FI = decltype(blocks)::value;
    f32x4 acc[FI][S::FJ];
    multiply<S, FI>(lds, feed, cur, following, at, [](int) { return 0; }, acc);
    at.younger = store_tile<S, FI, kLoadDefault>(
        lds, acc, g.out + (static_cast<int64_t>(t.start) + t.i0) * g.k + t.j * S::BJ, g.k, t.count - t.i0,
        g.k - t.j * S::BJ);
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

// ---- dw = dz^T x -----------------------------------------------------------------

// BI x BJ tiles of the experts' dw: the contraction runs over the expert's rows,
// none of them for an expert without rows (its dw is zeros).  An XCD takes one
// run of tiles, expert by expert: the expert's rows stay in its L2.
// PARTS: the rows of an expert are split into `parts` runs of whole steps, whose
// sums go to the workspace [parts][E][n][k] as fp32 and are added by join_kernel.
template <class S, bool PARTS>
__global__ __launch_bounds__(S::kThreads, S::kWavesPerSimd) void dw_kernel(ProductArgs g, int row_tiles, int total,
                                                                           int parts) {
  __shared__ __align__(1024) char smem[S::kLdsBytes];
  lds_ptr lds = (lds_ptr)smem;
  const int chunk = (total + 7) / 8, per = row_tiles * g.col_tiles;
  struct Tile {
    int e, i0, j0, part;
  };
  auto find = [&](int n) {
    Tile t{-1, 0, 0, 0};
    const int64_t pos = blockIdx.x / 8 + static_cast<int64_t>(n) * (gridDim.x / 8);
    int64_t id = (blockIdx.x % 8) * static_cast<int64_t>(chunk) + pos;
    if (pos >= chunk || id >= total) return t;
    if constexpr (PARTS) {
      t.part = static_cast<int>(id % parts);
      id /= parts;
    }
    t.e = static_cast<int>(id / per);
    const int q = static_cast<int>(id - static_cast<int64_t>(t.e) * per);
    const int group = q / (8 * g.col_tiles), rest = q - group * 8 * g.col_tiles;
    const int size = min(8, row_tiles - group * 8);
    t.j0 = rest / size * S::BJ;
    t.i0 = (group * 8 + rest % size) * S::BI;
    return t;
  };
  Tile t = find(0);
  if (t.e < 0) return;
  Feed<S, Across<S, S::BI, S::LI>, Across<S, S::BJ, S::LJ>, NoScaleLanes> feed;
  feed.i.init(g.n * 2);
  feed.j.init(g.k * 2);
  auto source = [&](const Tile &r) {
    Source s = kNoSource;
    if (r.e < 0) return s;
    ExpertRows rows = expert_rows(g.offsets, g.counts, r.e, g.rows);
    if constexpr (PARTS) {
      const int each = ((rows.count + parts - 1) / parts + kStepRows - 1) / kStepRows * kStepRows;
      const int first = min(r.part * each, rows.count);
      rows.start += first;
      rows.count = min(rows.count - first, each);
    }
    // the same in every lane: into scalar registers, where buffer resources live
    rows.start = __builtin_amdgcn_readfirstlane(rows.start);
    rows.count = __builtin_amdgcn_readfirstlane(rows.count);
    s.i = {reinterpret_cast<const char *>(g.dz + static_cast<int64_t>(rows.start) * g.n + r.i0), rows.count,
           r.i0 * 2};
    s.j = {reinterpret_cast<const char *>(g.x + static_cast<int64_t>(rows.start) * g.k + r.j0), rows.count,
           r.j0 * 2};
    s.steps = (rows.count + kStepRows - 1) / kStepRows;
    return s;
  };
  Source cur = source(t);
  start<S>(lds, feed, cur);
  Progress at;
  for (int n = 1; t.e >= 0; ++n) {
    const Tile next = find(n);
    const Source following = source(next);
    f32x4 acc[S::FI][S::FJ];
    multiply<S, S::FI>(lds, feed, cur, following, at, [](int) { return 0; }, acc);
    const int64_t row = static_cast<int64_t>(PARTS ? t.part * g.n_experts + t.e : t.e) * g.n + t.i0;
    if constexpr (PARTS)
      at.younger = store_tile<S, S::FI, kLoadDefault>(lds, acc, g.parts + row * g.k + t.j0, g.k, g.n - t.i0,
                                                      g.k - t.j0);
    else
      // streaming: what follows need not wait for dw to be written back (64 experts, 2048 x
      // 4096, 1 GB: 507 us against 538 for ordinary stores, and the next call's dz takes
      // 43 us, not 65; 256 MB: 113 against 142).  With a reader right behind, which might
      // have found dw in the caches, from 10% faster to 5% slower (m += c dw behind it,
      // 16 MB: 19.9 against 22.2 us, 64 MB 53.2 / 50.8, 128 MB 131.9 / 129.8, 256 MB 270 / 277,
      // 1 GB 1042 / 1078).
      at.younger =
          store_tile<S, S::FI, kLoadNT>(lds, acc, g.out + row * g.k + t.j0, g.k, g.n - t.i0, g.k - t.j0);
    t = next;
    cur = following;
  }
  wait_and_meet<0>();  // loads past the last tile fetch nothing, but write LDS
}

// dw from its parts, in their order: 8 values a thread.
__global__ __launch_bounds__(256) void join_kernel(ProductArgs g, int parts, int64_t vectors) {
  for (int64_t v = blockIdx.x * 256ll + threadIdx.x; v < vectors; v += gridDim.x * 256ll) {
    f32x4 lo{0.f, 0.f, 0.f, 0.f}, hi = lo;
    for (int q = 0; q < parts; ++q) {
      const f32x4 *from = reinterpret_cast<const f32x4 *>(g.parts + (q * vectors + v) * 8);
      lo += from[0];
      hi += from[1];
    }
    const float sum[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    store8(g.out + v * 8, sum);
  }
}

template <class S>
hipError_t launch_dx(ProductArgs g, int64_t pairs, hipStream_t stream) {
  g.col_tiles = (g.k + S::BJ - 1) / S::BJ;
  const int64_t tiles = row_tile_bound<S::BI>(pairs, g.n_experts) * g.col_tiles;
  if (tiles == 0) return hipSuccess;
  dx_kernel<S><<<tile_grid(tiles, S::kResident), S::kThreads, 0, stream>>>(g);
  return hipGetLastError();
}

template <class S>
hipError_t launch_dw(ProductArgs g, hipStream_t stream) {
  g.col_tiles = (g.k + S::BJ - 1) / S::BJ;
  const int row_tiles = (g.n + S::BI - 1) / S::BI;
  const int64_t total = static_cast<int64_t>(g.n_experts) * row_tiles * g.col_tiles;
  dw_kernel<S, false><<<tile_grid(total, S::kResident), S::kThreads, 0, stream>>>(g, row_tiles,
                                                                                 static_cast<int>(total), 1);
  return hipGetLastError();
}

template <class S>
hipError_t launch_dw_parts(ProductArgs g, int parts, hipStream_t stream) {
  g.col_tiles = (g.k + S::BJ - 1) / S::BJ;
  const int row_tiles = (g.n + S::BI - 1) / S::BI;
  const int64_t total = static_cast<int64_t>(g.n_experts) * row_tiles * g.col_tiles * parts;
  dw_kernel<S, true><<<tile_grid(total, S::kResident), S::kThreads, 0, stream>>>(g, row_tiles,
                                                                                static_cast<int>(total), parts);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t vectors = static_cast<int64_t>(g.n_experts) * g.n * g.k / 8, blocks = (vectors + 255) / 256;
  join_kernel<<<static_cast<uint32_t>(blocks < 4 * kComputeUnits ? blocks : 4 * kComputeUnits), 256, 0, stream>>>(
      g, parts, vectors);
  return hipGetLastError();
}

hipError_t launch_dx_sized(const ProductArgs &g, int64_t pairs, hipStream_t stream) {
  typedef Shape<256, 256, 2, 4, 2, false, true> Large;
  typedef Shape<128, 128, 2, 2, 2, false, true> Middle;
  typedef Shape<64, 128, 2, 2, 4, false, true> Small;
  // (Rounds of 256 workgroups, 256 x 256 against 128 x 128 tiles, us: 1.5 rounds, 24 experts
  // of 256 rows, K = 4096, N = 1024, 65.4 / 62.0, 12 of 1024, K = N = 2048, 103.9 / 99.1;
  // 2.0 rounds 77.0 / 94.4; 2.1 99.2 / 100.8; 3.5 139.5 / 155.3; 8, 64 experts of 384 rows,
  // K = 4096, N = 2048, 416 / 448.  Fewer: at kEnoughTiles.)
  if (row_tile_bound<Large::BI>(pairs, g.n_experts) * col_tiles<Large::BJ>(g.k) >= kEnoughTiles)
    return launch_dx<Large>(g, pairs, stream);
  if (row_tile_bound<Middle::BI>(pairs, g.n_experts) * col_tiles<Middle::BJ>(g.k) >= kEnoughTiles)
    return launch_dx<Middle>(g, pairs, stream);
  return launch_dx<Small>(g, pairs, stream);
}

// (2N = K = 1024: 8 experts, 128 tiles of 256 x 256, 31.6 us, of 128 x 128, 22.3;
// 16 experts, 256 tiles, 12.8 and 13.3; 2 experts with 2N = 512, K = 256 and 8192 rows,
// 16 tiles of 128 x 128, 79.7, of 64 x 64, 49.5.  The rows an expert has do not move the
// border, 256 x 256 / 128 x 128: 64 experts, 4096 x 2048, 64 rows 233 / 259, 128 rows 241 /
// 264, 384 rows 507 / 565, 1024 rows 1024 / 1215; 16 experts, 2048 x 2048, 256 tiles of
// 256 x 256: 37.0 / 35.7, 37.1 / 37.0, 65.4 / 65.1, 128.9 / 139.4.)
hipError_t launch_dw_sized(const ProductArgs &g, int parts, hipStream_t stream) {
  typedef Shape<256, 256, 2, 4, 2, true, true> Large;
  typedef Shape<128, 128, 2, 2, 2, true, true> Middle;
  typedef Shape<64, 64, 2, 2, 6, true, true> Small;
  if (parts > 1) return launch_dw_parts<Shape<kDwTile, kDwTile, 2, 2, 6, true, true>>(g, parts, stream);
  auto tiles = [&](auto shape) {
    typedef decltype(shape) S;
    return g.n_experts * col_tiles<S::BI>(g.n) * col_tiles<S::BJ>(g.k);
  };
  if (tiles(Large()) >= kComputeUnits) return launch_dw<Large>(g, stream);
  if (tiles(Middle()) >= kEnoughTiles) return launch_dw<Middle>(g, stream);
  return launch_dw<Small>(g, stream);
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
    const int64_t groups = expert_grad_workgroups(p, op.out_dim);
    err = glu ? launch_grad<true>(g, groups, op.act, stream) : launch_grad<false>(g, groups, op.act, stream);
    if (err != hipSuccess) return err;
    if (b.dbias) {
      bias_kernel<<<dim3((width + 15) / 16, p.n_experts), 256, 0, stream>>>(g, b.dbias);
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
  a.parts = nullptr;
  if (b.dx) {
    a.out = b.dx;
    err = launch_dx_sized(a, pairs, stream);
    if (err != hipSuccess) return err;
  }
  if (b.dw) {
    a.out = b.dw;
    a.parts = reinterpret_cast<float *>(static_cast<char *>(b.workspace) + expert_bias_bytes(p, op));
    err = launch_dw_sized(a, dw_parts(p, width, op.in_dim), stream);
  }
  return err;
}

}  // namespace moe
