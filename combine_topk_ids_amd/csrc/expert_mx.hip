// expert_mx.hip -- the experts' products with MX-FP4 weights over the packed rows (MX-FP4 or
// FP8):
//
//   gated block   z = x w_e^T + b_e (2F columns),  h = act(z[:F]) * z[F:]
//   linear layer  z = x w_e^T + b_e,               y = act(z) + residual
//
// Sums are fp32 accumulators of the scaled matrix instruction (mx_tile.hpp says what it keeps
// of its terms).  h and y are rounded once: to bf16, or h to MX-FP4 with the scale of
// its own 32 values, the rows of the next product.
//
// Few rows are bound by the weights' bytes (128 tokens, top 8 of 256 experts, K = 7168, F = 2048: 3.93
// GB in 638 us, 6.2 TB/s).  Many rows: a wave's reads of LDS and its products come one after the other
// (mx_tile.hpp), and the loads to LDS are issued late in a step (8192 tokens of the same layer:
// 1440-1460 us, 2.7 PFLOP/s, 7.3 GB fetched of 4.2; without loads 934).  FP8 rows: the same, with the
// matrix instructions in two halves and their vector work (24576 rows, K = 2048, N = 4096: 417 us,
// 346 without loads; those 65536 rows of K = 7168 3490-3620).
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
  if constexpr (GLU) feed.j.row.n = g.n;
  feed.i.init(x_bytes);
  feed.j.init(w_bytes);
  feed.s.init(x_scale_bytes, blocks, feed.j.row);
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
    constexpr int kHalves = GLU ? 2 : 1;             // blocks of z to one of y
    constexpr int kPairs = S::FJ / kHalves / 2;      // of blocks of y
    static_assert(kPairs * 2 * kHalves == S::FJ, "y leaves by pairs of blocks");
    f32x4 acc[FI][S::FJ];
    multiply_mx<S, FI>(lds, feed, cur, following, blocks, at, acc);
    const int lane = late_lane_id();
    if constexpr (S::WK > 1) {
      // the groups' sums, added in order by the first
      lds_ptr sums = (lds_ptr)smem + S::WK * S::kGroupLds + lane * 16;
      if (group_id<S>() > 0) {
#pragma unroll
        for (int b = 0; b < S::FJ; ++b)
          *(MOE_LDS f32x4 *)(sums + (group_id<S>() - 1) * S::kSums + b * kWave * 16) = acc[0][b];
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
          acc[0][b] += *(MOE_LDS const f32x4 *)(sums + (q - 1) * S::kSums + b * kWave * 16);
    }
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
    // A lane has 4 neighbouring columns of each block of y.  Lanes 16 apart exchange those of two
    // blocks, and each has 8 of one: 16 bytes of bf16, a quarter of the pair's 32 columns.
    const int i_lane = lane & 15, quarter = lane >> 4;
    const int col_lane = col0 + (quarter & 1) * 16 + (quarter >> 1) * 8;
    // place of the lane's values of pair h, block row a: past the results' end kNowhere
    auto place = [&](int a, int h) {
      const int i = (w.wi + a * S::WI) * 16 + i_lane, col = col_lane + h * 32;
      return i < left && col < g.n ? static_cast<uint32_t>(i * g.n + col) : kNowhere;
    };
    auto in_bytes = [](uint32_t at) { return static_cast<int>(at == kNowhere ? at : at * 2); };
    // all of the residual before the first store: one trip to memory
    uint4 add[GLU ? 1 : FI][kPairs];
    if constexpr (!GLU) {
      if (g.residual) {
        const auto r = buffer_rsrc(g.residual + row0 * g.n, kRecords);
#pragma unroll
        for (int a = 0; a < FI; ++a)
#pragma unroll
          for (int h = 0; h < kPairs; ++h)
            add[a][h] = __builtin_bit_cast(
                uint4, __builtin_amdgcn_raw_buffer_load_b128(r, in_bytes(place(a, h)), 0, kLoadDefault));
      }
    }
    auto leave = [&](auto act) {
      constexpr int ACT = decltype(act)::value;
#pragma unroll
      for (int a = 0; a < FI; ++a) {
#pragma unroll
        for (int b = 0; b < S::FJ; ++b) acc[a][b] += shift[b];
#pragma unroll
        for (int h = 0; h < kPairs; ++h) {
          float v[8];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t y[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int b = (h * 2 + u) * kHalves;
              y[u] = __float_as_uint(act_value<ACT>(acc[a][b][c]) * (GLU ? acc[a][b + kHalves - 1][c] : 1.0f));
            }
            // odd rows of 16 lanes of the first change places with even rows of the second
            const auto p = __builtin_amdgcn_permlane16_swap(y[0], y[1], false, false);
            const uint32_t x0 = p[0], x1 = p[1];
            v[c] = __uint_as_float(x0);
            v[c + 4] = __uint_as_float(x1);
          }
          const uint32_t to = place(a, h);
          if (GLU && g.codes) {
            // a row's 32 columns are in four lanes, 16 apart
            uint32_t am = mx_lane_max(v);
            const auto p = __builtin_amdgcn_permlane16_swap(am, am, false, false);
            am = max(static_cast<uint32_t>(p[0]), static_cast<uint32_t>(p[1]));
            const auto p2 = __builtin_amdgcn_permlane32_swap(am, am, false, false);
            am = max(static_cast<uint32_t>(p2[0]), static_cast<uint32_t>(p2[1]));
            uint32_t scale;
            const uint32_t c = mx_encode8(v, am, scale);  // (n is a multiple of 32: whole blocks are in or out)
            const auto rc = buffer_rsrc(g.codes + row0 * (g.n / 2), kRecords);
            const auto rs = buffer_rsrc(g.scales + row0 * (g.n / 32), kRecords);
            __builtin_amdgcn_raw_buffer_store_b32(c, rc, static_cast<int>(to == kNowhere ? to : to / 2), 0, 0);
            const bool leads = to != kNowhere && quarter == 0;
            __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(scale), rs,
                                                 static_cast<int>(leads ? to / 32 : kNowhere), 0, 0);
          } else {
            if constexpr (!GLU) {
              if (g.residual) {
                float more[8];
                unpack8(add[a][h], more);
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] += more[c];
              }
            }
            store8(buffer_rsrc(g.y + row0 * g.n, kRecords), static_cast<uint32_t>(in_bytes(to)), v);
          }
        }
      }
    };
    switch (g.act) {
      case MOE_ACT_SILU: leave(std::integral_constant<int, MOE_ACT_SILU>()); break;
      case MOE_ACT_GELU_TANH: leave(std::integral_constant<int, MOE_ACT_GELU_TANH>()); break;
      case MOE_ACT_RELU: leave(std::integral_constant<int, MOE_ACT_RELU>()); break;
      default: leave(std::integral_constant<int, MOE_ACT_NONE>());
    }
    at.younger = FI * kPairs;
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
hipError_t launch(MxArgs g, int64_t pairs, hipStream_t stream, int resident = S::kResident) {
  constexpr int kCols = GLU ? S::BJ / 2 : S::BJ;
  g.col_tiles = (g.n + kCols - 1) / kCols;
  const int64_t tiles = row_tile_bound<S::BI>(pairs, g.n_experts) * g.col_tiles;
  mx_kernel<S, GLU><<<tile_grid(tiles, resident), S::kThreads * S::WK, 0, stream>>>(g);
  return hipGetLastError();
}

// Which tile, by the rows an expert has on average, the contraction's length and whether larger
// tiles would leave compute units without work.  MX-FP4 rows: 128 x 128 and, for many rows, 256 x 256.
// FP8 rows, whose split into two halves is vector work that a wave does once for all its columns:
// 64 x 128 in four waves of 16 x 128, and 128 x 256 in eight of 32 x 128 (that in waves of 64 x 64:
// 24576 rows, K = 2048, N = 4096, 64 experts 451 us against 390).  Measured, us a call, gated, K = 4096,
// F = 1024, 64 experts:
//   rows an expert           0.1     4*     12**   16     24     48    128    192    384***
//   16 x 64, K in four       8.5   600.2    80.2   65.0   82.1  127.6  300.4  441.5  1724
//   16 x 64                 15.8   613.0    56.0   63.7   80.8  130.9  312.3  475.0  2073
//   128 x 128               14.7   678.2    61.8   54.8   55.6   60.4   89.5  104.4   329
//   256 x 256               21.0   829.8    71.4   64.1   65.3   67.8   79.3   90.9   276
//   FP8: 16 x 64, K in four 11.2   909.6           92.7         145.6^        690.9
//        16 x 64            20.2   640.2           78.7         110.7^        520.2
//        64 x 128           27.6   887.5           69.6          72.7^        225.2
//        128 x 256          54.1  1406.3          109.8         110.4^        213.0
// (* K = 7168, F = 2048, 256 experts; ** linear, K = 2048, N = 4096; *** F = 2048; ^ 32 rows; 96: 133.8
// of 64 x 128, 114.4 of 128 x 256.)
// A tile of 16 rows is one wave with two stages, so that a compute unit holds six and the
// weights, which pass once, never wait for one barrier (three stages a wave, four waves with a common
// one: 926 us for 640 above).  Where tiles are few the time is that of one chain of steps, and a long
// contraction goes to the four waves of a workgroup.
// A short contraction does not pay for 256 x 256's first loads and last stores (256 rows, N = 4096, 128
// x 128 and 256 x 256: K = 512 58.4 / 61.9, 1024 80.6 / 80.8, 2048 130.8 / 124.1; linear, N = 7168, K = 1024
// 83.2 / 92.1), nor does one whose rows (K / 2 bytes) start inside a line: of each the two lines
// that a step touches come twice, more often than the caches keep them (256 rows, N = 4096,
// K = 4128 306 / 460).
// The average is all that the host knows: where a routing sends every row to a few experts, the tile
// for few rows reads their weights once for every 16 rows (gated, K = 4096, F = 1024, 171 rows on each of
// six experts: of 256 37 us, with the tile for many rows, which a layer of six gets, 16.6).
template <bool GLU, bool FP8, bool ODD>
hipError_t launch_sized(const MxArgs &g, int64_t pairs, hipStream_t stream) {
  typedef MxShape<16, 64, 1, 1, FP8 ? 2 : 3, FP8, ODD, true, 4> Split;
  typedef MxShape<16, 64, 1, 1, 2, FP8, ODD, true> Few;
  typedef typename std::conditional<FP8, MxShape<64, 128, 4, 1, 2, FP8, ODD, false>,
                                    MxShape<128, 128, 2, 2, 2, FP8, ODD, false>>::type Some;
  typedef typename std::conditional<FP8, MxShape<128, 256, 4, 2, 2, FP8, ODD, false>,
                                    MxShape<256, 256, 2, 4, 2, FP8, ODD, false>>::type Many;
  const int64_t used = pairs < g.n_experts ? pairs : g.n_experts, rows = (pairs + used - 1) / used;
  const int wrows = g.n * (GLU ? 2 : 1);
  const int64_t split_tiles = row_tile_bound<Split::BI>(pairs, g.n_experts) * col_tiles<Split::BJ>(wrows);
  const int64_t many_tiles = row_tile_bound<Many::BI>(pairs, g.n_experts) * col_tiles<Many::BJ>(wrows);
  if (g.k >= 2048 && split_tiles <= 2 * kComputeUnits) return launch<Split, GLU>(g, pairs, stream);
  if (rows <= 12) return launch<Few, GLU>(g, pairs, stream);
  if constexpr (!ODD) {
    const bool deep = FP8 || g.k >= 1536;
    if (rows > (FP8 ? 80 : 112) && deep && many_tiles >= kEnoughTiles) return launch<Many, GLU>(g, pairs, stream);
  }
  return launch<Some, GLU>(g, pairs, stream);
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
