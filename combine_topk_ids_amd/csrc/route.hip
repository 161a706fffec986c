// route.hip -- routing: scores, top-k experts and gate weights from a router's logits,
// and the gradient of the weights and scores with respect to the logits.
//
//   s = softmax(l) or sigmoid(l);  experts in order of s + bias (of l without a bias);
//   w_j = scale * s_j, or scale * s_j / sum_i s_i over the chosen ones
//
// A token is a run of L lanes of a wave (16, 32 or 64), each with PER neighbouring experts
// in registers; the k <= L choices end one to a lane.  Keys are compared as whole numbers in
// the values' order.  The order of two experts must not hang on a rounding.  Without a bias it is
// that of the logits, which is exact.  With one, and for sums of two in a group, values are formed
// in fp32 first; where two that are told apart lie nearer than their errors could
// move them, the wave forms all of them again in 64 bits (8192 tokens, 256 experts, 8 groups and a
// bias: 13.5-14.4 us, 64 bits for every token 29.6).
//
// Bound by vector instructions (770 a wave of that case) and, for few tokens, by the chain of
// k + 1 reductions over the lanes: 4.7 us for one token, 6.1 for 16384 of 128 bf16 logits, whose 5 MB
// are one.
#include <initializer_list>
#include <type_traits>

#include "moe_device.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

// a or b, as values: of two array elements `c ? a : b` chooses the place, and what follows
// from that is an array indexed by a register, resolved with a chain of selects at every use.
template <class V>
__device__ __forceinline__ V pick(bool c, V a, V b) {
  return c ? a : b;
}

// What the wave's lanes wrote to LDS before is what they read after.  (LDS serves a wave in order;
// this keeps the compiler to it: no instruction.)
__device__ __forceinline__ void lanes_meet() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// -------------------------------------------------- a token's lanes ---

// f(v of a lane, v of its partner) over the L lanes of a token, in a fixed order: every
// lane ends with the same bits.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// v of this lane and of the lane STEP away, in either order (f is symmetric).
template <int STEP>
__device__ __forceinline__ u32x2 both(uint32_t v) {
  if constexpr (STEP == 1) return u32x2{v, dpp<kQuadSwap1>(v)};
  if constexpr (STEP == 2) return u32x2{v, dpp<kQuadSwap2>(v)};
  if constexpr (STEP == 4) return u32x2{v, dpp<kRowHalfMirror>(v)};
  if constexpr (STEP == 8) return u32x2{v, dpp<kRowMirror>(v)};
  // odd rows (the upper half) of the first change places with even rows (the lower half) of the second
  if constexpr (STEP == 16) return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
}
template <int STEP, class V, class F>
__device__ __forceinline__ V with_partner(V v, F f) {
  if constexpr (sizeof(V) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const u32x2 lo = both<STEP>(static_cast<uint32_t>(b)), hi = both<STEP>(static_cast<uint32_t>(b >> 32));
    return f(__builtin_bit_cast(V, static_cast<uint64_t>(hi.x) << 32 | lo.x),
             __builtin_bit_cast(V, static_cast<uint64_t>(hi.y) << 32 | lo.y));
  } else {
    const u32x2 p = both<STEP>(__builtin_bit_cast(uint32_t, v));
    const uint32_t x = p.x, y = p.y;  // (a cast of a vector's element takes the first one)
    return f(__builtin_bit_cast(V, x), __builtin_bit_cast(V, y));
  }
}
template <int L, class V, class F>
__device__ __forceinline__ V all_lanes(V v, F f) {
  v = with_partner<1>(v, f);
  v = with_partner<2>(v, f);
  v = with_partner<4>(v, f);
  v = with_partner<8>(v, f);
  if constexpr (L >= 32) v = with_partner<16>(v, f);
  if constexpr (L >= 64) v = with_partner<32>(v, f);
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

// v of a lane that holds what the lane STEP away does.
template <int STEP, class V>
__device__ __forceinline__ V partner(V v) {
  auto one = [](uint32_t u) {
    const u32x2 p = both<STEP>(u);
    const uint32_t x = p.x, y = p.y;
    return STEP >= 16 && (lane_id() & STEP) ? x : y;
  };
  if constexpr (sizeof(V) == 8)
    return static_cast<V>(one(static_cast<uint32_t>(v >> 32))) << 32 | one(static_cast<uint32_t>(v));
  else
    return one(v);
}

// v of a lane of the token (the same number in every lane).
template <int L, class V>
__device__ __forceinline__ V lane_value(V v, int lane) {
  auto one = [&](uint32_t u) -> uint32_t {
    if constexpr (L == kWave) return __builtin_amdgcn_readlane(u, lane);
    return __shfl(static_cast<int>(u), lane, L);
  };
  if constexpr (sizeof(V) == 8)
    return static_cast<V>(one(static_cast<uint32_t>(v >> 32))) << 32 | one(static_cast<uint32_t>(v));
  else
    return one(v);
}

// ---------------------------------------------------------- keys ---

// Whole numbers in the order of the values: above 0 (not to be chosen) for every value
// but -inf; both zeros alike; a NaN above all.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t key = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return pick(v != v, 0xFFFFFFFFu, pick(v == -kInf, 0u, key));
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  const uint64_t key = u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 1ull << 63);
  return pick(v != v, ~uint64_t{0}, pick(v == -__builtin_inf(), uint64_t{0}, key));
}

// exp, off by at most (3 + 0.23 |x|) 2^-24 of itself: the hardware's exp2 (a unit in the last place), a last
// rounding, and what log2 e loses as an fp32 number (1.93e-8, times |x| ln 2).  The rounding of
// the argument's product is put right.  Zero below 2^-126.
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
// A sigmoid s and 1 - s, both to a few units in the last place, for the slope s (1 - s): taken from a
// rounded s near 1 the complement has lost its bits (l = 12: 2%, 14: 11%, from 17 on all).
struct SigmoidParts {
  float s, rest;
};
__device__ __forceinline__ SigmoidParts sigmoid_parts(float l) {
  const float t = exp_fine(-fabsf(l)), large = __builtin_amdgcn_rcpf(1.0f + t), small = t * large;
  return {pick(l < 0.0f, small, large), pick(l < 0.0f, large, small)};
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

// Softmax of a row held PER to a lane: v becomes exp(l - top), top the row's maximum; the result is
// their sum's reciprocal (0 for a row of -inf; NaN where a NaN or +inf is in the row).
template <int L, int PER>
__device__ __forceinline__ float softmax_parts(const float (&l)[PER], float (&v)[PER], float &top) {
  top = -kInf;
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

// The value of a key (that of -0 is +0).
__device__ __forceinline__ float key_value(uint32_t u) {
  return u == 0xFFFFFFFFu ? __builtin_nanf("") : __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ double key_value(uint64_t u) {
  return u == ~0ull ? __builtin_nan("") : __builtin_bit_cast(double, u ^ (u >> 63 ? 1ull << 63 : ~0ull));
}

// Whether fp32 values a >= b could be the other way round, or equal: `slack` is what the errors of
// two scores (or of two sums of two) can come to, 2^-21 what the additions round.
// A sigmoid is off by at most 4.2 * 2^-24 (exp_fine's error weighs s (1 - s), at most 1/4, or 0.224 with
// the factor |l|; the sum and the reciprocal 1.5 * 2^-23 s), four of them by 2^-19.  A softmax score
// s = e^x / sum, x = l - top: its exponential is off by (3 + 1.3 |x|) 2^-24 of itself (the
// rounding of x too), which is at most 3 s + 1.3 / e in all, as s |x| <= 1 / e; the sum by
// 33 * 2^-24 of itself (its terms' mean |x| is at most log 1024, so 12, and 21 additions),
// the reciprocal and the product by 2.  Scores of a row add up to 1 at most: four of them by
// (3 + 35 + 4 * 1.3 / e) 2^-24 = 40 * 2^-24, less than 2^-18.  (A NaN or two infinities are not near: a score
// with its bias never overflows, so neither becomes another value in 64 bits.)
constexpr float kSigmoidSlack = 0x1p-19f, kSoftmaxSlack = 0x1p-18f;
__device__ __forceinline__ bool too_near(float a, float b, float slack) {
  return a - b <= slack + 0x1p-21f * fabsf(a);
}

// The k largest keys of a token, best first; lane j gets the expert of the j-th, -1 where
// none is left.  near (in some lane of the token): two neighbours in that order, the first left
// out among them, are too near to tell (fp32 keys that stand for others).
//
// A lane sorts its four keys once (a stable network), and offers its best; of the lanes that
// have the largest the one with the lowest index gives it up: two reductions a choice, and no
// more than five registers change.  (More keys a lane: it looks for its best again each time.)
template <int L, int PER, bool NEAR, class K>
__device__ __forceinline__ int choose(K (&key)[PER], int k, float slack, bool &near) {
  const int lane = lane_id() & (L - 1);
  constexpr bool kSorted = PER <= 4;
  int slot[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) slot[i] = lane * PER + i;
  if constexpr (kSorted) {
#pragma unroll
    for (int n = PER - 1; n > 0; --n)
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const bool swap = key[i + 1] > key[i];
        const K high = pick(swap, key[i + 1], key[i]), low = pick(swap, key[i], key[i + 1]);
        const int first = pick(swap, slot[i + 1], slot[i]), second = pick(swap, slot[i], slot[i + 1]);
        key[i] = high;
        key[i + 1] = low;
        slot[i] = first;
        slot[i + 1] = second;
      }
  }
  int mine = -1;
  K own = 0, last = 0;
  for (int j = 0; j < k + (NEAR ? 1 : 0); ++j) {
    K best = key[0];
    int at = slot[0];
    if constexpr (!kSorted) {
#pragma unroll
      for (int i = 1; i < PER; ++i) {
        const bool more = key[i] > best;
        best = pick(more, key[i], best);
        at = pick(more, slot[i], at);
      }
    }
    const K top = lanes_best<L>(best);
    if constexpr (NEAR) {
      if (j == k) {  // the first left out
        near = near || (top != 0 && too_near(key_value(last), key_value(top), slack));
        break;
      }
      last = top;
    }
    int id;
    bool gives;  // (with nothing left: a key of 0 becomes 0)
    if constexpr (L == kWave) {
      const int who = __builtin_ctzll(ballot(best == top));
      id = __builtin_amdgcn_readlane(at, who);
      gives = lane == who;
    } else {
      const int offer = best == top ? at : 0x7FFFFFFF;
      id = all_lanes<L>(offer, [](int a, int b) { return a < b ? a : b; });
      gives = offer == id;
    }
    if (lane == j) {
      mine = top != 0 ? id : -1;
      own = top;
    }
    if constexpr (kSorted) {
#pragma unroll
      for (int i = 0; i + 1 < PER; ++i) {
        key[i] = pick(gives, key[i + 1], key[i]);
        slot[i] = pick(gives, slot[i + 1], slot[i]);
      }
      key[PER - 1] = pick(gives, K{0}, key[PER - 1]);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = pick(gives && slot[i] == id, K{0}, key[i]);
    }
  }
  if constexpr (NEAR) {
    // lane j holds the j-th key: each against the one before it
    const K before = static_cast<K>(__shfl_up(static_cast<int>(own), 1, L));
    near = near || (lane > 0 && lane < k && own != 0 && too_near(key_value(before), key_value(own), slack));
  }
  return lane < k ? mine : -1;
}

// As choose(), of keys whose upper halves alone count (bf16 logits): the lower half takes the
// expert's index, so that one reduction finds key and expert, and nothing else moves along.
// (16384 tokens, 128 experts, top 8: 7.6 us with choose().)
template <int L, int PER>
__device__ __forceinline__ int choose_short(const uint32_t (&key)[PER], int k) {
  const int lane = lane_id() & (L - 1);
  uint32_t v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    v[i] = pick(key[i] == 0, 0u, (key[i] & 0xFFFF0000u) | (0xFFFFu - static_cast<uint32_t>(lane * PER + i)));
  constexpr bool kSorted = PER <= 4;
  if constexpr (kSorted) {
#pragma unroll
    for (int n = PER - 1; n > 0; --n)
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const uint32_t a = v[i], b = v[i + 1];
        v[i] = max(a, b);
        v[i + 1] = min(a, b);
      }
  }
  uint32_t mine = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = v[0];
    if constexpr (!kSorted) {
#pragma unroll
      for (int i = 1; i < PER; ++i) best = max(best, v[i]);
    }
    const uint32_t top = lanes_best<L>(best);
    if (lane == j) mine = top;
    if constexpr (kSorted) {
      const bool gives = best == top;
#pragma unroll
      for (int i = 0; i + 1 < PER; ++i) v[i] = pick(gives, v[i + 1], v[i]);
      v[PER - 1] = pick(gives, 0u, v[PER - 1]);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = pick(v[i] == top, 0u, v[i]);
    }
  }
  return lane < k && mine != 0 ? static_cast<int>(0xFFFFu - (mine & 0xFFFFu)) : -1;
}

// A group's key from its two best (0: none): the best, or with `two` the sum's.  error: what the
// roundings of two biased scores and of their sum, each by 2^-24, and of adding this to it come to:
// the two can cancel, so it goes by them and not by the sum.
__device__ __forceinline__ uint32_t group_key(uint32_t first, uint32_t second, bool two, float &error) {
  const float a = key_value(first);
  error = first != 0 ? 0x1p-22f * fabsf(a) : 0.0f;
  if (!two || second == 0) return first;
  const float b = key_value(second), sum = a + b;
  error += 0x1p-22f * fabsf(b);
  // (a sum below all numbers is still one that can be chosen)
  return order_key(pick(sum == -kInf, -__FLT_MAX__, sum));
}
__device__ __forceinline__ uint64_t group_key(uint64_t first, uint64_t second, bool two, float &) {
  return two && second != 0 ? order_key(key_value(first) + key_value(second)) : first;
}

// Keys of experts outside the best groups become 0.  value: the key of an expert's part of its
// group's score, 0 if it cannot be chosen.  `row`: an LDS row of L * PER keys.
template <int L, int PER, bool NEAR, class V, class K>
__device__ __forceinline__ void keep_groups(const RouteArgs &g, const V (&value)[PER], uint64_t *lds_row,
                                            K (&key)[PER], float slack, bool &near) {
  const int lane = lane_id() & (L - 1), e0 = lane * PER;
  const bool two = g.group_top == 2;
  // of the lane's own groups: the lowest that a kept one can be, the highest of one left out
  // (past the largest number a NaN, which settles nothing below)
  V kept = static_cast<V>(~0ull), out = 0;
  auto place = [&](V mine, float error, int better) {
    const bool keep = better < g.top_groups;
    if constexpr (NEAR) {
      const V at = mine == 0 ? 0 : order_key(key_value(mine) + (keep ? -error : error));
      if (keep)
        kept = at < kept ? at : kept;
      else
        out = at > out ? at : out;
    }
    return keep;
  };
  // lanes that hold a group, where it is a power of two of them
  const int group_lanes = g.group_size % PER ? 0 : g.group_size / PER;
  if (group_lanes > 0 && (group_lanes & (group_lanes - 1)) == 0) {
    V first = 0, second = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const V low = pick(value[i] < first, value[i], first);
      first = pick(value[i] > first, value[i], first);
      second = pick(low > second, low, second);
    }
    auto merge = [&](auto step) {
      constexpr int STEP = decltype(step)::value;
      if (group_lanes <= STEP) return;
      const V a = partner<STEP>(first), b = partner<STEP>(second);
      const V low = pick(a < first, a, first), high = pick(second > b, second, b);
      first = pick(a > first, a, first);
      second = pick(low > high, low, high);
    };
    merge(std::integral_constant<int, 1>());
    merge(std::integral_constant<int, 2>());
    merge(std::integral_constant<int, 4>());
    merge(std::integral_constant<int, 8>());
    if constexpr (L >= 32) merge(std::integral_constant<int, 16>());
    if constexpr (L >= 64) merge(std::integral_constant<int, 32>());
    float error = 0.0f;
    const V mine = group_key(first, second, two, error);
    const int own = lane / group_lanes;
    int better = 0;
    for (int h = 0; h < g.groups; ++h) {
      const V u = lane_value<L>(mine, h * group_lanes);
      better += u > mine || (u == mine && h < own);
    }
    if (own < g.groups && !place(mine, error, better)) {
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = 0;
    }
  } else {
    V *row = reinterpret_cast<V *>(lds_row);
    lanes_meet();
#pragma unroll
    for (int i = 0; i < PER; ++i) row[e0 + i] = value[i];
    lanes_meet();
    // a group's key takes the place of its first expert's, the error the next
    for (int q = lane; q < g.groups; q += L) {
      V first = 0, second = 0;
      for (int i = 0; i < g.group_size; ++i) {
        const V u = row[q * g.group_size + i];
        const V low = u < first ? u : first;
        first = u > first ? u : first;
        second = low > second ? low : second;
      }
      float error = 0.0f;
      row[q * g.group_size] = group_key(first, second, two, error);
      if constexpr (NEAR) {
        if (g.group_size > 1) row[q * g.group_size + 1] = __float_as_uint(error);
      }
    }
    lanes_meet();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = e0 + i;
      if (e < g.e) {
        const int q = e / g.group_size;
        const V mine = row[q * g.group_size];
        int better = 0;
        for (int h = 0; h < g.groups; ++h) {
          const V u = row[h * g.group_size];
          better += u > mine || (u == mine && h < q);
        }
        float error = 0.0f;
        if constexpr (NEAR)
          error = g.group_size > 1 ? __uint_as_float(row[q * g.group_size + 1])
                                   : 0x1p-22f * fabsf(key_value(mine));
        if (!place(mine, error, better)) key[i] = 0;
      }
    }
    lanes_meet();
  }
  if constexpr (NEAR) {
    kept = ~lanes_best<L>(static_cast<V>(~kept));
    out = lanes_best<L>(out);
    if (out != 0) near = near || !(key_value(kept) - key_value(out) > slack);
  }
}

// The choices of token t by a whole wave, in 64 bits: lane j gets the j-th expert.
template <int PER, class T>
__device__ __forceinline__ int choose64(const RouteArgs &g, int64_t t, uint64_t *lds_row) {
  const int e0 = lane_id() * PER;
  float l[PER], b[PER];
  load_row(static_cast<const T *>(g.logits) + t * g.e, e0, g.e, false, -kInf, l);
#pragma unroll
  for (int i = 0; i < PER; ++i) b[i] = 0.0f;
  if (g.bias) load_row(g.bias, e0, g.e, false, 0.0f, b);
  double v[PER];
  scores64<kWave>(l, g.sigmoid, v);
  uint64_t part[PER], key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    part[i] = l[i] == -kInf ? 0 : order_key(v[i] + b[i]);
    key[i] = g.bias ? part[i] : order_key(static_cast<double>(l[i]));
  }
  bool ignored = false;
  if (g.groups > 1) keep_groups<kWave, PER, false>(g, part, lds_row, key, 0.0f, ignored);
  return choose<kWave, PER, false>(key, g.k, 0.0f, ignored);
}

template <int L, int PER, class T>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs g) {
  constexpr int kTokens = kThreads / L;
  __shared__ uint64_t rows[kThreads * PER];
  const int lane = lane_id() & (L - 1), e0 = lane * PER, own = threadIdx.x / L;
  uint64_t *mine = rows + own * L * PER;
  const bool sums = g.groups > 1 && g.group_top == 2;
  float b[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) b[i] = 0.0f;
  if (g.bias) load_row(g.bias, e0, g.e, g.vector, 0.0f, b);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const bool live = t0 + own < g.n;
  const int64_t t = live ? t0 + own : t0;
  const T *row = static_cast<const T *>(g.logits) + t * g.e;
  float l[PER];
  load_row(row, e0, g.e, g.vector, -kInf, l);

  // scores, where something besides the chosen logits needs them
  float s[PER], inv = 1.0f, top = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) s[i] = 0.0f;
  if (g.sigmoid) {
    if (g.scores || g.bias || sums) {
#pragma unroll
      for (int i = 0; i < PER; ++i) s[i] = sigmoid_fine(l[i]);
    }
  } else if (g.scores || g.bias || sums || !g.renormalize) {
    inv = softmax_parts<L>(l, s, top);
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] *= inv;
  }
  if (g.scores && live) store_row(g.scores + t * g.e, e0, g.e, g.vector, s);

  uint32_t key[PER];
  bool near = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = order_key(l[i]);  // 0: not to be chosen
  auto choose_logits = [&](uint32_t(&of)[PER]) {
    if constexpr (sizeof(T) == 2)
      return choose_short<L, PER>(of, g.k);
    else
      return choose<L, PER, false>(of, g.k, 0.0f, near);
  };
  int id;
  if (g.bias || sums) {
    const float slack = g.sigmoid ? kSigmoidSlack : kSoftmaxSlack;
    uint32_t part[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) part[i] = pick(key[i] == 0, 0u, order_key(s[i] + b[i]));
    if (g.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = part[i];
    }
    if (g.groups > 1) keep_groups<L, PER, true>(g, part, mine, key, slack, near);
    id = g.bias ? choose<L, PER, true>(key, g.k, slack, near) : choose_logits(key);
    // again in 64 bits, a token at a time
    const int first = threadIdx.x / kWave * kWave / L;  // the wave's first token in the workgroup
    for (int q = 0; q < kWave / L; ++q) {
      const uint64_t m = ballot(near && live && own - first == q);
      if (m == 0) continue;
      const int other = choose64<PER * L / kWave, T>(g, t0 + first + q, rows + first * L * PER);
      const int same = __shfl(other, lane);
      if (own - first == q) id = same;
    }
  } else {
    if (g.groups > 1) {
      uint32_t part[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) part[i] = key[i];
      keep_groups<L, PER, false>(g, part, mine, key, 0.0f, near);
    }
    id = choose_logits(key);
  }

  if (lane < g.k && live) g.ids[t * g.k + lane] = id;
  if (!g.weights) return;
  // lane j: the j-th choice's logit and weight
  float w = 0.0f;
  const bool held = lane < g.k && id >= 0;
  float chosen = -kInf;
  if (held) chosen = load_one(row + id);
  if (g.sigmoid) {
    w = held ? sigmoid_fine(chosen) : 0.0f;
  } else if (g.renormalize) {
    float best = lanes_max<L>(chosen);
    if (best == -kInf) best = 0.0f;
    w = held ? exp_fine(chosen - best) : 0.0f;
  } else {
    w = held ? exp_fine(chosen - top) * inv : 0.0f;  // the score's bits
  }
  if (g.renormalize) {
    const float sum = lanes_sum<L>(w);
    w = sum == 0.0f ? 0.0f : w / sum;
  }
  if (held && inv != inv) w = inv;  // a NaN among the token's logits
  if (lane < g.k && live) g.weights[t * g.k + lane] = w * g.scale;
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

// Softmax: dl = s (d - sum d s); sigmoid: dl = d s (1 - s); renormalised weights w = s / sum s of
// the chosen: u_j = w_j (d_j - sum d w), times 1 - s_j for a sigmoid.  Read and written once, so
// bound by the latency of one token's loads: 16384 tokens, 128 experts, bf16, both gradients 6.6 us
// for 17.8 MB; 333 tokens of 60 3.3.
template <int L, int PER, class T>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteGradArgs g) {
  constexpr int kTokens = kThreads / L;
  __shared__ float rows[kThreads * PER];
  const int lane = lane_id() & (L - 1), e0 = lane * PER, own = threadIdx.x / L;
  float *add = rows + own * L * PER;
  // whether a gradient reaches experts that were not chosen
  const bool whole = g.dscores || (!g.sigmoid && !g.renormalize);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
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
    SigmoidParts sj{0.0f, 0.0f};
    if (g.sigmoid && held) sj = sigmoid_parts(chosen);
    if (g.renormalize) {
      float w = sj.s;
      if (!g.sigmoid) {
        float top = lanes_max<L>(chosen);
        if (top == -kInf) top = 0.0f;
        w = held ? exp_fine(chosen - top) : 0.0f;
      }
      const float sum = lanes_sum<L>(w);
      w = sum == 0.0f ? 0.0f : w / sum;
      const float dot = lanes_sum<L>(u * w);
      u = held ? w * (u - dot) : 0.0f;
      if (g.sigmoid) u *= sj.rest;
    } else if (g.sigmoid) {
      u *= sj.s * sj.rest;
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
    lanes_meet();
    if (first) add[id] = total;
    lanes_meet();
  }
  float out[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) out[i] = add[e0 + i];
  lanes_meet();
  if (whole) {
    if (g.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const SigmoidParts p = sigmoid_parts(l[i]);
        out[i] += d[i] * (p.s * p.rest);
      }
    } else {
      float top;
      const float inv = softmax_parts<L>(l, s, top);
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

// f(integral_constant<L>, integral_constant<PER>): the lanes of a token and the experts of
// a lane that E experts and k choices need.  The choice is bound by its instructions, of which
// whole waves with four keys a lane need the fewest past 128 experts (8192 tokens,
// 256 experts: 16 lanes of 16 keys 24.8 us, 64 of 4 16.5); the gradient by its loads, of which few
// lanes have more in flight (16384 tokens, 128 experts: 16 lanes of 8 6.3 us, 32 of 4 7.5).
template <bool BACKWARD, class F>
hipError_t with_lanes(int e, int k, F f) {
  typedef std::integral_constant<int, 4> Four;
  typedef std::integral_constant<int, 8> Eight;
  typedef std::integral_constant<int, 16> Sixteen;
  typedef std::integral_constant<int, 64> All;
  if (e <= 64 && k <= 16) return f(Sixteen(), Four());
  if constexpr (BACKWARD) {
    if (e <= 128 && k <= 16) return f(Sixteen(), Eight());
    if (e <= 256 && k <= 16) return f(Sixteen(), Sixteen());
  } else {
    if (e <= 128 && k <= 32) return f(std::integral_constant<int, 32>(), Four());
  }
  if (e <= 256) return f(All(), Four());
  if (e <= 512) return f(All(), Eight());
  return f(All(), Sixteen());
}

// Tokens of one launch (a launch's threads fit 32 bits): more take several.
constexpr int64_t kLaunchTokens = 1 << 22;

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
  g.group_top = r.group_top;
  g.sigmoid = r.score == MOE_SCORE_SIGMOID;
  g.renormalize = r.renormalize != 0;
  g.vector = whole_vectors(g.e, {scores, bias}, {logits}, bf16);
  g.scale = r.scale;
  return with_lanes<false>(g.e, g.k, [&](auto l, auto per) {
    constexpr int L = decltype(l)::value, PER = decltype(per)::value, kTokens = kThreads / L;
    for (int64_t from = 0; from < p.n_tokens; from += kLaunchTokens) {
      RouteArgs part = g;
      part.n = p.n_tokens - from < kLaunchTokens ? p.n_tokens - from : kLaunchTokens;
      part.logits = static_cast<const char *>(logits) + from * g.e * (bf16 ? 2 : 4);
      part.ids += from * g.k;
      if (weights) part.weights += from * g.k;
      if (scores) part.scores += from * g.e;
      const uint32_t grid = static_cast<uint32_t>((part.n + kTokens - 1) / kTokens);
      if (bf16)
        route_kernel<L, PER, uint16_t><<<grid, kThreads, 0, stream>>>(part);
      else
        route_kernel<L, PER, float><<<grid, kThreads, 0, stream>>>(part);
    }
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
  return with_lanes<true>(g.e, g.k, [&](auto l, auto per) {
    constexpr int L = decltype(l)::value, PER = decltype(per)::value, kTokens = kThreads / L;
    for (int64_t from = 0; from < p.n_tokens; from += kLaunchTokens) {
      RouteGradArgs part = g;
      part.n = p.n_tokens - from < kLaunchTokens ? p.n_tokens - from : kLaunchTokens;
      part.logits = static_cast<const char *>(logits) + from * g.e * (bf16 ? 2 : 4);
      part.dlogits = static_cast<char *>(dlogits) + from * g.e * (bf16 ? 2 : 4);
      if (ids) part.ids += from * g.k;
      if (dweights) part.dweights += from * g.k;
      if (dscores) part.dscores += from * g.e;
      const uint32_t grid = static_cast<uint32_t>((part.n + kTokens - 1) / kTokens);
      if (bf16)
        route_backward_kernel<L, PER, uint16_t><<<grid, kThreads, 0, stream>>>(part);
      else
        route_backward_kernel<L, PER, float><<<grid, kThreads, 0, stream>>>(part);
    }
    return hipGetLastError();
  });
}

}  // namespace moe
