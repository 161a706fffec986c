// route.hip -- routing: scores, top-k experts and gate weights from a router's logits,
// and the gradient of the weights and scores with respect to the logits.
//
//   s = softmax(l) or sigmoid(l);  experts in order of s + bias (of l without a bias);
//   w_j = scale * s_j, or scale * s_j / sum_i s_i over the chosen ones
//
// A token is a run of L lanes of a wave (16 or 64), each with PER neighbouring experts
// in registers; the k <= L choices end one to a lane.  The order of two experts must
// not hang on a rounding, so keys are compared as whole numbers: without a bias the logits'
// own bits, with one the bits of s + bias in 64 bits.
#include <initializer_list>
#include <type_traits>

#include "moe_device.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

// -------------------------------------------------- a token's lanes ---

template <int L>
__device__ __forceinline__ uint32_t other(uint32_t v, int step) {
  return static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), step));
}

// f(v of a lane, v of its partner) over the L lanes of a token, in a fixed order: every
// lane ends with the same bits.
template <int L, class V, class F>
__device__ __forceinline__ V all_lanes(V v, F f) {
  auto with = [&](auto move) {
    if constexpr (sizeof(V) == 8) {
      const uint64_t b = __builtin_bit_cast(uint64_t, v);
      const uint64_t lo = move(static_cast<uint32_t>(b)), hi = move(static_cast<uint32_t>(b >> 32));
      v = f(v, __builtin_bit_cast(V, hi << 32 | lo));
    } else {
      v = f(v, __builtin_bit_cast(V, move(__builtin_bit_cast(uint32_t, v))));
    }
  };
  with([](uint32_t b) { return dpp<kQuadSwap1>(b); });
  with([](uint32_t b) { return dpp<kQuadSwap2>(b); });
  with([](uint32_t b) { return dpp<kRowHalfMirror>(b); });
  with([](uint32_t b) { return dpp<kRowMirror>(b); });
  if constexpr (L == 64) {
    with([](uint32_t b) { return other<L>(b, 16); });
    with([](uint32_t b) { return other<L>(b, 32); });
  }
  return v;
}
template <int L, class V>
__device__ __forceinline__ V lanes_sum(V v) {
  return all_lanes<L>(v, [](V a, V b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  return all_lanes<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L, class K>
__device__ __forceinline__ K lanes_best(K v) {
  return all_lanes<L>(v, [](K a, K b) { return a > b ? a : b; });
}

// Lowest lane of this token for which p holds, counted from its first; -1: none.
template <int L>
__device__ __forceinline__ int first_lane(bool p) {
  uint64_t m = ballot(p);
  if constexpr (L < kWave) m = (m >> (lane_id() & ~(L - 1))) & ((1ull << L) - 1);
  return m ? __builtin_ctzll(m) : -1;
}

// ---------------------------------------------------------- keys ---

// Whole numbers in the order of the values: above 0 (not to be chosen) for every value
// but -inf; both zeros alike; a NaN above all.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  if (v == -kInf) return 0;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return ~0ull;
  if (v == -__builtin_inf()) return 0;
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return u ^ (u >> 63 ? ~0ull : 1ull << 63);
}

// exp to about one unit in the last place (the hardware's exp2 with the argument's
// rounding put right); zero below 2^-126.
__device__ __forceinline__ float exp_fine(float x) {
  constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
  const float t = x * kLog2e;
  const float y = __builtin_amdgcn_exp2f(t);
  const float rest = __builtin_fmaf(x, kLog2e, -t);  // NaN for an infinite t
  return fabsf(rest) < 1.0f && y < kInf ? __builtin_fmaf(y, rest * kLn2, y) : y;
}
__device__ __forceinline__ float sigmoid_fine(float l) {
  return __builtin_amdgcn_rcpf(1.0f + exp_fine(-l));
}

// ---------------------------------------------------------- rows ---

struct RouteArgs {
  const void *logits;
  const float *bias;
  int32_t *ids;
  float *weights, *scores;
  int64_t n;
  int e, k, groups, group_size, top_groups, group_top;
  bool sigmoid, renormalize, vector;  // vector: rows are whole 16-byte pieces
  float scale;
};

// PER values of a row from column e0 on; past the row's end `none`.
template <int PER>
__device__ __forceinline__ void load_row(const float *row, int e0, int e, bool vector, float none,
                                         float (&v)[PER]) {
  if (vector) {
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const bool in = e0 + i < e;
      const float4 f = in ? *reinterpret_cast<const float4 *>(row + e0 + i) : float4{none, none, none, none};
      v[i] = f.x;
      v[i + 1] = f.y;
      v[i + 2] = f.z;
      v[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = e0 + i < e ? row[e0 + i] : none;
  }
}
template <int PER>
__device__ __forceinline__ void load_row(const uint16_t *row, int e0, int e, bool vector, float none,
                                         float (&v)[PER]) {
  if (vector) {  // 4 at a time: rows are whole 8-byte pieces
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const bool in = e0 + i < e;
      const uint2 w = in ? *reinterpret_cast<const uint2 *>(row + e0 + i) : uint2{0, 0};
      v[i] = in ? bf16_lo(w.x) : none;
      v[i + 1] = in ? bf16_hi(w.x) : none;
      v[i + 2] = in ? bf16_lo(w.y) : none;
      v[i + 3] = in ? bf16_hi(w.y) : none;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      v[i] = e0 + i < e ? __uint_as_float(static_cast<uint32_t>(row[e0 + i]) << 16) : none;
  }
}
template <int PER>
__device__ __forceinline__ void store_row(float *row, int e0, int e, bool vector, const float (&v)[PER]) {
  if (vector) {
#pragma unroll
    for (int i = 0; i < PER; i += 4)
      if (e0 + i < e) *reinterpret_cast<float4 *>(row + e0 + i) = float4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < e) row[e0 + i] = v[i];
  }
}
template <int PER>
__device__ __forceinline__ void store_row(uint16_t *row, int e0, int e, bool vector, const float (&v)[PER]) {
  if (vector) {
#pragma unroll
    for (int i = 0; i < PER; i += 4)
      if (e0 + i < e)
        *reinterpret_cast<uint2 *>(row + e0 + i) =
            uint2{f32_to_bf16(v[i]) | f32_to_bf16(v[i + 1]) << 16,
                  f32_to_bf16(v[i + 2]) | f32_to_bf16(v[i + 3]) << 16};
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < e) row[e0 + i] = static_cast<uint16_t>(f32_to_bf16(v[i]));
  }
}

__device__ __forceinline__ float load_one(const float *p) { return *p; }
__device__ __forceinline__ float load_one(const uint16_t *p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

// Softmax of a row held PER to a lane: v becomes exp(l - max), the result is their
// sum's reciprocal (0 for a row of -inf; NaN where a NaN or +inf is in the row).
template <int L, int PER>
__device__ __forceinline__ float softmax_parts(const float (&l)[PER], float (&v)[PER]) {
  float top = -kInf;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
  top = lanes_max<L>(top);
  if (top == -kInf) top = 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = exp_fine(l[i] - top);
    sum += v[i];
  }
  sum = lanes_sum<L>(sum);
  return sum == 0.0f ? 0.0f : 1.0f / sum;
}

// Scores in 64 bits.
template <int L, int PER>
__device__ __forceinline__ void scores64(const float (&l)[PER], bool sigmoid, double (&s)[PER]) {
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = 1.0 / (1.0 + exp(-static_cast<double>(l[i])));
    return;
  }
  float top = -kInf;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
  top = lanes_max<L>(top);
  if (top == -kInf) top = 0.0f;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    s[i] = exp(static_cast<double>(l[i]) - top);
    sum += s[i];
  }
  sum = lanes_sum<L>(sum);
#pragma unroll
  for (int i = 0; i < PER; ++i) s[i] = sum == 0.0 ? 0.0 : s[i] / sum;
}

// ----------------------------------------------------- selection ---

// The k largest keys of a token, best first; lane j gets the expert of the j-th, -1 where
// none is left.
template <int L, int PER, class K>
__device__ __forceinline__ int choose(K (&key)[PER], int k) {
  const int lane = lane_id() & (L - 1);
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    K best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool more = key[i] > best;
      best = more ? key[i] : best;
      at = more ? i : at;
    }
    const K top = lanes_best<L>(best);
    const int who = first_lane<L>(best == top && top != 0);  // the lowest index of the best
    const int slot = __shfl(at, who < 0 ? 0 : who, L);
    if (lane == j) mine = who < 0 ? -1 : who * PER + slot;
    if (lane == who) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == slot) key[i] = 0;
    }
  }
  return mine;
}

// Keys of experts outside the best groups become 0.  value: an expert's part of its
// group's score, -inf if it cannot be chosen.  `row`: an LDS row of L * PER keys.
template <int L, int PER, class K>
__device__ __forceinline__ void keep_groups(const RouteArgs &g, const double (&value)[PER], uint64_t *row,
                                            K (&key)[PER]) {
  const int lane = lane_id() & (L - 1), e0 = lane * PER;
  auto of = [](uint64_t u) {
    return u == ~0ull ? __builtin_nan("") : __builtin_bit_cast(double, u ^ (u >> 63 ? 1ull << 63 : ~0ull));
  };
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < PER; ++i) row[e0 + i] = order_key(value[i]);
  __builtin_amdgcn_wave_barrier();
  // a group's key takes the place of its first expert's
  for (int q = lane; q < g.groups; q += L) {
    uint64_t first = 0, second = 0;
    for (int i = 0; i < g.group_size; ++i) {
      const uint64_t u = row[q * g.group_size + i];
      if (u > first) {
        second = first;
        first = u;
      } else if (u > second) {
        second = u;
      }
    }
    if (g.group_top == 2 && second != 0) first = order_key(of(first) + of(second));
    row[q * g.group_size] = first;
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i;
    if (e < g.e) {
      const int q = e / g.group_size;
      const uint64_t mine = row[q * g.group_size];
      int better = 0;
      for (int h = 0; h < g.groups; ++h) {
        const uint64_t u = row[h * g.group_size];
        better += u > mine || (u == mine && h < q);
      }
      if (better >= g.top_groups) key[i] = 0;
    }
  }
  __builtin_amdgcn_wave_barrier();
}

template <int L, int PER, class T>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs g) {
  constexpr int kTokens = kThreads / L;
  __shared__ uint64_t rows[kThreads * PER];
  const int lane = lane_id() & (L - 1), e0 = lane * PER, own = threadIdx.x / L;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTokens;
  // (whole waves go round together)
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens; t0 < g.n; t0 += stride) {
    const bool live = t0 + own < g.n;
    const int64_t t = live ? t0 + own : t0;
    const T *row = static_cast<const T *>(g.logits) + t * g.e;
    float l[PER];
    load_row(row, e0, g.e, g.vector, -kInf, l);

    // scores, where something besides the chosen logits needs them
    float s[PER], inv = 1.0f;
    const bool stats = g.scores || g.bias || !g.renormalize || g.sigmoid;
    if (g.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) s[i] = sigmoid_fine(l[i]);
    } else if (stats) {
      inv = softmax_parts<L>(l, s);
#pragma unroll
      for (int i = 0; i < PER; ++i) s[i] *= inv;
    }
    if (g.scores && live) store_row(g.scores + t * g.e, e0, g.e, g.vector, s);

    uint64_t *mine = rows + own * L * PER;
    const bool sums = g.groups > 1 && g.group_top == 2;
    double v[PER];
    if (g.bias || sums) {
      float b[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) b[i] = 0.0f;
      if (g.bias) load_row(g.bias, e0, g.e, false, -kInf, b);
      scores64<L>(l, g.sigmoid, v);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        v[i] = l[i] == -kInf || e0 + i >= g.e ? -__builtin_inf() : v[i] + b[i];
    }
    int id;
    if (g.bias) {
      uint64_t key[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = order_key(v[i]);
      if (g.groups > 1) keep_groups<L>(g, v, mine, key);
      id = choose<L>(key, g.k);
    } else {
      uint32_t key[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = order_key(l[i]);
      if (g.groups > 1) {
        if (!sums) {
#pragma unroll
          for (int i = 0; i < PER; ++i) v[i] = l[i];
        }
        keep_groups<L>(g, v, mine, key);
      }
      id = choose<L>(key, g.k);
    }

    if (lane < g.k && live) g.ids[t * g.k + lane] = id;
    if (!g.weights) continue;
    // lane j: the j-th choice's logit and weight
    float w = 0.0f;
    const bool held = lane < g.k && id >= 0;
    float chosen = -kInf;
    if (held) chosen = load_one(row + id);
    if (g.sigmoid) {
      w = held ? sigmoid_fine(chosen) : 0.0f;
    } else if (g.renormalize) {
      float top = lanes_max<L>(chosen);
      if (top == -kInf) top = 0.0f;
      w = held ? exp_fine(chosen - top) : 0.0f;
    } else {
      // the same bits as the score's
      float top = -kInf;
#pragma unroll
      for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
      top = lanes_max<L>(top);
      if (top == -kInf) top = 0.0f;
      w = held ? exp_fine(chosen - top) * inv : 0.0f;
    }
    if (g.renormalize) {
      const float sum = lanes_sum<L>(w);
      w = sum == 0.0f ? 0.0f : w / sum;
    }
    if (held && inv != inv) w = inv;  // a NaN among the token's logits
    if (lane < g.k && live) g.weights[t * g.k + lane] = w * g.scale;
  }
}

// ------------------------------------------------------ gradient ---

struct RouteGradArgs {
  const void *logits;
  const int32_t *ids;
  const float *dweights, *dscores;
  void *dlogits;
  int64_t n;
  int e, k;
  bool sigmoid, renormalize, vector;
  float scale;
};

template <int L, int PER, class T>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteGradArgs g) {
  constexpr int kTokens = kThreads / L;
  __shared__ float rows[kThreads * PER];
  const int lane = lane_id() & (L - 1), e0 = lane * PER, own = threadIdx.x / L;
  float *add = rows + own * L * PER;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTokens;
  // whether a gradient reaches experts that were not chosen
  const bool whole = g.dscores || (!g.sigmoid && !g.renormalize);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens; t0 < g.n; t0 += stride) {
    const bool live = t0 + own < g.n;
    const int64_t t = live ? t0 + own : t0;
    const T *row = static_cast<const T *>(g.logits) + t * g.e;
    float l[PER], s[PER], d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = d[i] = 0.0f;
    if (whole) {
      load_row(row, e0, g.e, g.vector, -kInf, l);
      if (g.dscores) load_row(g.dscores + t * g.e, e0, g.e, g.vector, 0.0f, d);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) add[e0 + i] = 0.0f;
    if (g.dweights) {
      // lane j: the j-th choice
      int id = lane < g.k ? g.ids[t * g.k + lane] : -1;
      const bool held = id >= 0 && id < g.e;
      if (!held) id = -1;
      float u = held ? g.dweights[t * g.k + lane] * g.scale : 0.0f;
      float chosen = -kInf;
      if (held) chosen = load_one(row + id);
      const float sj = g.sigmoid && held ? sigmoid_fine(chosen) : 0.0f;
      if (g.renormalize) {
        float w = sj;
        if (!g.sigmoid) {
          float top = lanes_max<L>(chosen);
          if (top == -kInf) top = 0.0f;
          w = held ? exp_fine(chosen - top) : 0.0f;
        }
        const float sum = lanes_sum<L>(w);
        w = sum == 0.0f ? 0.0f : w / sum;
        const float dot = lanes_sum<L>(u * w);
        u = held ? w * (u - dot) : 0.0f;
        if (g.sigmoid) u *= 1.0f - sj;
      } else if (g.sigmoid) {
        u *= sj * (1.0f - sj);
      }
      // an ID that repeats within the token: its first lane adds up all
      float total = 0.0f;
      bool first = held;
      for (int j = 0; j < g.k; ++j) {
        const int other_id = __shfl(id, j, L);
        const float other_u = __shfl(u, j, L);
        if (other_id == id) {
          total += other_u;
          if (j < lane) first = false;
        }
      }
      __builtin_amdgcn_wave_barrier();
      if (first) add[id] = total;
      __builtin_amdgcn_wave_barrier();
    }
    float out[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) out[i] = add[e0 + i];
    __builtin_amdgcn_wave_barrier();
    if (whole) {
      if (g.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const float p = sigmoid_fine(l[i]);
          out[i] += d[i] * p * (1.0f - p);
        }
      } else {
        const float inv = softmax_parts<L>(l, s);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          s[i] *= inv;
          if (!g.renormalize) {
            d[i] += out[i];
            out[i] = 0.0f;
          }
          dot += e0 + i < g.e ? d[i] * s[i] : 0.0f;
        }
        dot = lanes_sum<L>(dot);
#pragma unroll
        for (int i = 0; i < PER; ++i) out[i] += s[i] * (d[i] - dot);
      }
    }
    if (live) store_row(static_cast<T *>(g.dlogits) + t * g.e, e0, g.e, g.vector, out);
  }
}

// f(integral_constant<L>, integral_constant<PER>): the lanes of a token and the experts of
// a lane that E experts and k choices need.
template <class F>
hipError_t with_lanes(int e, int k, F f) {
  auto at = [&](auto l, auto per) { return f(l, per); };
  typedef std::integral_constant<int, 4> Four;
  typedef std::integral_constant<int, 8> Eight;
  typedef std::integral_constant<int, 16> Sixteen;
  typedef std::integral_constant<int, 64> All;
  if (k <= 16 && e <= 256) {
    if (e <= 64) return at(Sixteen(), Four());
    if (e <= 128) return at(Sixteen(), Eight());
    return at(Sixteen(), Sixteen());
  }
  if (e <= 256) return at(All(), Four());
  if (e <= 512) return at(All(), Eight());
  return at(All(), Sixteen());
}

// Workgroups: a round of the whole device at most, which then go on.
constexpr int64_t kMostBlocks = 1 << 20;
inline uint32_t token_blocks(int64_t n, int tokens) {
  const int64_t b = (n + tokens - 1) / tokens;
  return static_cast<uint32_t>(b < kMostBlocks ? b : kMostBlocks);
}

// Rows of e values that start, like the arrays, on whole vectors of four.
inline bool whole_vectors(int e, std::initializer_list<const void *> f32, std::initializer_list<const void *> t,
                          bool bf16) {
  bool ok = e % 4 == 0;
  for (const void *p : f32) ok = ok && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  for (const void *p : t) ok = ok && reinterpret_cast<uintptr_t>(p) % (bf16 ? 8 : 16) == 0;
  return ok;
}

}  // namespace

hipError_t launch_route(const moe_problem &p, const moe_router &r, const void *logits, const float *bias,
                        int32_t *ids, float *weights, float *scores, hipStream_t stream) {
  if (p.n_tokens == 0) return hipSuccess;
  const bool bf16 = r.logits == MOE_LOGITS_BF16;
  RouteArgs g;
  g.logits = logits;
  g.bias = bias;
  g.ids = ids;
  g.weights = weights;
  g.scores = scores;
  g.n = p.n_tokens;
  g.e = p.n_experts;
  g.k = p.top_k;
  g.groups = r.top_groups < r.n_groups ? r.n_groups : 1;  // all groups kept: no choice to make
  g.group_size = p.n_experts / g.groups;
  g.top_groups = r.top_groups;
  // (a group of one expert has no second)
  g.group_top = r.group_top;
  g.sigmoid = r.score == MOE_SCORE_SIGMOID;
  g.renormalize = r.renormalize != 0;
  g.vector = whole_vectors(g.e, {scores}, {logits}, bf16);
  g.scale = r.scale;
  return with_lanes(g.e, g.k, [&](auto l, auto per) {
    constexpr int L = decltype(l)::value, PER = decltype(per)::value;
    const uint32_t grid = token_blocks(g.n, kThreads / L);
    if (bf16)
      route_kernel<L, PER, uint16_t><<<grid, kThreads, 0, stream>>>(g);
    else
      route_kernel<L, PER, float><<<grid, kThreads, 0, stream>>>(g);
    return hipGetLastError();
  });
}

hipError_t launch_route_backward(const moe_problem &p, const moe_router &r, const void *logits,
                                 const int32_t *ids, const float *dweights, const float *dscores,
                                 void *dlogits, hipStream_t stream) {
  if (p.n_tokens == 0) return hipSuccess;
  const bool bf16 = r.logits == MOE_LOGITS_BF16;
  RouteGradArgs g;
  g.logits = logits;
  g.ids = ids;
  g.dweights = dweights;
  g.dscores = dscores;
  g.dlogits = dlogits;
  g.n = p.n_tokens;
  g.e = p.n_experts;
  g.k = p.top_k;
  g.sigmoid = r.score == MOE_SCORE_SIGMOID;
  g.renormalize = r.renormalize != 0;
  g.vector = whole_vectors(g.e, {dscores}, {logits, dlogits}, bf16);
  g.scale = r.scale;
  return with_lanes(g.e, g.k, [&](auto l, auto per) {
    constexpr int L = decltype(l)::value, PER = decltype(per)::value;
    const uint32_t grid = token_blocks(g.n, kThreads / L);
    if (bf16)
      route_backward_kernel<L, PER, uint16_t><<<grid, kThreads, 0, stream>>>(g);
    else
      route_backward_kernel<L, PER, float><<<grid, kThreads, 0, stream>>>(g);
    return hipGetLastError();
  });
}

}  // namespace moe
