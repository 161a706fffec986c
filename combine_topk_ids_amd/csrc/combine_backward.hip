// combine_backward.hip -- gradients of the combine
//
//   out[t] = sum_j w[t][j] * Y[slot[t][j]]
//   dY[slot[t][j]] = bf16(w[t][j] * dout[t])        (one fp32 product, rounded once)
//   dw[t][j] = <Y[slot[t][j]], dout[t]>             (fp32 sum)
//
// Memory bound: dout is read once per token, each expert row read once and
// each gradient row written once.  One workgroup of four waves per token (or, for
// rows of at most 512 columns, one wave); the waves take the token's 512-column
// chunks in turn (8 columns a lane) and keep the k dot products in registers; at the
// end the lanes' sums are added in a fixed order, so runs repeat bit for bit.
// Measured: 8192 tokens, k = 8, H = 7168: 400 us, 4.9 TB/s, what a copy reaches.  A
// masked slot (or one outside the rows) gets a buffer resource of zero bytes: its
// loads return zeros and its stores are dropped by the hardware, with no branch
// between the chunk's loads.  A token's rows are its own (slots are distinct), so no
// two workgroups write one row.
#include "moe_device.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kBatch = 8;  // slots handled together when k is not a compile-time constant

struct CombineGradArgs {
  const uint16_t *y, *dout;
  const int32_t *slot;
  const float *w;
  uint16_t *dy;
  float *dw;
  int64_t n, rows;
  int k, h;
};

__device__ __forceinline__ void widen(const u32x4 v, float (&f)[8]) {
  unpack8(__builtin_bit_cast(uint4, v), f);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// KC > 0: k is the compile-time constant KC.  WPT: waves of a token, 4 or 1.
template <int KC, int WPT>
__global__ __launch_bounds__(kWaves *kWave) void combine_backward_kernel(CombineGradArgs g) {
  constexpr int KB = KC > 0 ? KC : kBatch;
  __shared__ float part[kWaves][KB];
  constexpr int kTokens = kWaves / WPT;  // of a workgroup at a time
  const int id = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int wave = WPT == 1 ? 0 : id;
  const int k = KC > 0 ? KC : g.k, nvec = g.h / 8;
  const uint32_t row_bytes = 2u * static_cast<uint32_t>(g.h);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + (WPT == 1 ? id : 0); t < g.n;
       t += static_cast<int64_t>(gridDim.x) * kTokens) {
    const int64_t pair0 = t * k;
    const int my_slot = lane < k ? g.slot[pair0 + lane] : -1;
    const float my_w = lane < k ? (g.w ? g.w[pair0 + lane] : 1.0f) : 0.0f;
    const auto rd = buffer_rsrc(g.dout + t * g.h, row_bytes);
    for (int j0 = 0; j0 < k; j0 += KB) {
      float acc[KB];
      uint32_t bytes[KB];
      int64_t at[KB];
      float wj[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int s = j0 + j < k ? __builtin_amdgcn_readlane(my_slot, j0 + j) : -1;
        const bool live = s >= 0 && s < g.rows;
        bytes[j] = live ? row_bytes : 0u;
        at[j] = live ? static_cast<int64_t>(s) * g.h : 0;
        wj[j] = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_w), j0 + j < k ? j0 + j : 0));
        acc[j] = 0.0f;
      }
      for (int v = wave * kWave; v < nvec; v += WPT * kWave) {
        const int off = (v + lane) * 16;  // past the row: no access
        const u32x4 dv = __builtin_amdgcn_raw_buffer_load_b128(rd, off, 0, kLoadDefault);
        u32x4 yv[KB];
        if (g.dw) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            yv[j] = __builtin_amdgcn_raw_buffer_load_b128(buffer_rsrc(g.y + at[j], bytes[j]), off, 0,
                                                          kLoadDefault);
        }
        float d[8];
        widen(dv, d);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          u32x4 o;
          o.x = f32_to_bf16(wj[j] * d[0]) | (f32_to_bf16(wj[j] * d[1]) << 16);
          o.y = f32_to_bf16(wj[j] * d[2]) | (f32_to_bf16(wj[j] * d[3]) << 16);
          o.z = f32_to_bf16(wj[j] * d[4]) | (f32_to_bf16(wj[j] * d[5]) << 16);
          o.w = f32_to_bf16(wj[j] * d[6]) | (f32_to_bf16(wj[j] * d[7]) << 16);
          __builtin_amdgcn_raw_buffer_store_b128(o, buffer_rsrc(g.dy + at[j], bytes[j]), off, 0, 0);
        }
        if (g.dw) {
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            float y[8];
            widen(yv[j], y);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[j] = __builtin_fmaf(y[c], d[c], acc[j]);
          }
        }
      }
      if (!g.dw) continue;
      // a masked pair has no row: its gradient is zero, whatever dout holds
      if constexpr (WPT == 1) {
        float mine = 0.0f;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const float s = wave_sum(acc[j]);
          if (lane == j && bytes[j]) mine = s;
        }
        if (lane < KB && j0 + lane < k) g.dw[pair0 + j0 + lane] = mine;
      } else {
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const float s = wave_sum(acc[j]);
          if (lane == 0) part[wave][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < KB && j0 + static_cast<int>(threadIdx.x) < k) {
          const int j = threadIdx.x, s = g.slot[pair0 + j0 + j];
          const float v = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
          g.dw[pair0 + j0 + j] = s >= 0 && s < g.rows ? v : 0.0f;
        }
        __syncthreads();
      }
    }
  }
}

template <int WPT>
hipError_t launch_k(const CombineGradArgs &g, hipStream_t stream) {
  const int64_t groups = (g.n + kWaves / WPT - 1) / (kWaves / WPT);
  const dim3 grid(static_cast<uint32_t>(groups < (1 << 20) ? groups : 1 << 20)), threads(kWaves * kWave);
  switch (g.k) {
    case 1: combine_backward_kernel<1, WPT><<<grid, threads, 0, stream>>>(g); break;
    case 2: combine_backward_kernel<2, WPT><<<grid, threads, 0, stream>>>(g); break;
    case 4: combine_backward_kernel<4, WPT><<<grid, threads, 0, stream>>>(g); break;
    case 6: combine_backward_kernel<6, WPT><<<grid, threads, 0, stream>>>(g); break;
    case 8: combine_backward_kernel<8, WPT><<<grid, threads, 0, stream>>>(g); break;
    default: combine_backward_kernel<0, WPT><<<grid, threads, 0, stream>>>(g); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_backward(const moe_problem &p, const moe_plan &plan, const uint16_t *expert_out,
                                   const float *weights, const uint16_t *dout, uint16_t *dy,
                                   float *dweights, hipStream_t stream) {
  if (p.n_tokens == 0) return hipSuccess;
  CombineGradArgs g;
  g.y = expert_out;
  g.dout = dout;
  g.slot = plan.slot;
  g.w = weights;
  g.dy = dy;
  g.dw = dweights;
  g.n = p.n_tokens;
  g.rows = max_rows(p);
  g.k = p.top_k;
  g.h = p.hidden;
  // rows of at most one wave's 512 columns: a token a wave (H = 88, k = 2, 14297 tokens:
  // 9.0 us against 17.9); wider ones: four waves a token, also where one wave would
  // do as well, for the tokens' latency when they are few
  if (p.hidden <= 8 * kWave) return launch_k<1>(g, stream);
  return launch_k<kWaves>(g, stream);
}

}  // namespace moe
