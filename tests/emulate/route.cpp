// Routing, its gradient and MX-FP4 quantisation, lane by lane on the CPU, over random sizes: every
// load and store inside its array, and the results right.
//
// Arguments: seed, cases.
#define kThreads kQuantizeThreads
#include "quantize.inc"
#undef kThreads
#include "route.inc"

#include <memory>
#include <numeric>

namespace moe {
namespace {

std::mt19937 draw(1);
int upto(int n) { return static_cast<int>(draw() % n); }
double normal() {
  static std::normal_distribution<double> d;
  return d(draw);
}

// n values in memory that ends where they end
template <class T>
std::unique_ptr<T[]> array(size_t n) {
  return std::unique_ptr<T[]>(new T[n]());
}

struct Case {
  moe_problem p;
  moe_router r;
  bool bias, scores, weights;
  int kind;  // logits: 0 normal, 1 ties, 2 switched-off experts, 3 wide
};

Case any() {
  Case c{};
  const int groups = upto(2) ? 1 : 1 << upto(4);
  int each = 1 + upto(upto(4) ? 24 : 1024 / groups);
  if (upto(2)) each = std::min((each + 3) / 4 * 4, 1024 / groups);  // rows of whole vectors
  c.p.n_experts = groups * each;
  c.r.n_groups = groups;
  c.r.top_groups = 1 + upto(groups);
  c.r.group_top = 1 + upto(2);
  c.p.top_k = 1 + upto(std::min(upto(3) ? 8 : 64, c.r.top_groups * each));
  c.p.n_tokens = 1 + upto(upto(2) ? 5 : 40);
  c.p.hidden = 8;
  c.p.ep = 1;
  c.p.pad_multiple = 1;
  c.r.score = upto(2);
  c.r.logits = upto(2);
  c.r.renormalize = upto(2);
  c.r.scale = upto(2) ? 1.0f : 2.5f;
  c.bias = upto(2);
  c.scores = upto(2);
  c.weights = upto(8);
  c.kind = upto(4);
  return c;
}

// what a row's logits are held in
float rounded(double v, bool bf16) {
  const float f = static_cast<float>(v);
  return bf16 ? __uint_as_float(f32_to_bf16(f) << 16) : f;
}

struct Token {
  std::vector<double> s, away;  // scores; 1 - s
};
Token token(const float *l, int e, bool sigmoid) {
  Token t{std::vector<double>(e), std::vector<double>(e)};
  double top = -INFINITY, sum = 0;
  for (int i = 0; i < e; ++i) top = std::max(top, static_cast<double>(l[i]));
  for (int i = 0; i < e; ++i) sum += std::isinf(l[i]) ? 0 : std::exp(l[i] - top);
  for (int i = 0; i < e; ++i) {
    if (sigmoid) {
      t.s[i] = 1 / (1 + std::exp(-static_cast<double>(l[i])));
      t.away[i] = 1 / (1 + std::exp(static_cast<double>(l[i])));
    } else {
      t.s[i] = std::isinf(l[i]) ? 0 : std::exp(l[i] - top) / sum;
      t.away[i] = 1 - t.s[i];
    }
  }
  return t;
}

std::vector<int> choices(const Case &c, const float *l, const float *bias, const Token &t) {
  const int e = c.p.n_experts, each = e / c.r.n_groups;
  std::vector<double> part(e), key(e);
  for (int i = 0; i < e; ++i) {
    part[i] = std::isinf(l[i]) ? -INFINITY : t.s[i] + (bias ? static_cast<double>(bias[i]) : 0);
    key[i] = bias ? part[i] : l[i];
  }
  auto best = [](const std::vector<double> &v) {
    std::vector<int> order(v.size());
    std::iota(order.begin(), order.end(), 0);
    std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return v[a] > v[b]; });
    return order;
  };
  if (c.r.top_groups < c.r.n_groups) {
    std::vector<double> total(c.r.n_groups);
    for (int q = 0; q < c.r.n_groups; ++q) {
      const double *from = (c.r.group_top == 2 ? part : key).data() + q * each;
      std::vector<double> v(from, from + each);
      std::sort(v.begin(), v.end(), std::greater<double>());
      total[q] = v[0] + (c.r.group_top == 2 && each > 1 && !std::isinf(v[1]) ? v[1] : 0);
    }
    const std::vector<int> order = best(total);
    for (int q = c.r.top_groups; q < c.r.n_groups; ++q)
      std::fill(key.begin() + order[q] * each, key.begin() + (order[q] + 1) * each, -INFINITY);
  }
  std::vector<int> ids = best(key);
  ids.resize(c.p.top_k);
  for (int &id : ids)
    if (std::isinf(key[id])) id = -1;
  return ids;
}

void close(double got, double want, double far, const char *what) {
  if (std::abs(got - want) <= far) return;
  fprintf(stderr, "%s: %.9g, wanted %.9g, may be off by %g\n", what, got, want, far);
  emu::fail("a wrong result");
}

void one(const Case &c) {
  const int n = static_cast<int>(c.p.n_tokens), e = c.p.n_experts, k = c.p.top_k;
  const bool bf16 = c.r.logits == MOE_LOGITS_BF16, sigmoid = c.r.score == MOE_SCORE_SIGMOID;
  printf("tokens %d experts %d k %d groups %d of %d by %d, score %d bf16 %d renormalize %d bias %d scores %d kind %d\n",
         n, e, k, c.r.top_groups, c.r.n_groups, c.r.group_top, c.r.score, bf16, c.r.renormalize, c.bias, c.scores, c.kind);
  fflush(stdout);
  if (host::check_router(&c.p, &c.r) != MOE_OK) emu::fail("a refused case");
  // (one past a whole vector now and then)
  const int skip = upto(4) ? 0 : 1 + upto(3);
  auto l = array<float>(n * e);
  auto held = array<float>(skip + (bf16 ? 0 : n * e));
  auto held16 = array<uint16_t>(skip + (bf16 ? n * e : 0));
  for (int i = 0; i < n * e; ++i) {
    double v = normal();
    if (c.kind == 1) v = std::round(v * 2) / 2;
    if (c.kind == 2 && upto(5) < 2) v = -INFINITY;
    if (c.kind == 3) v *= 12;
    l[i] = rounded(v, bf16);
    if (bf16)
      held16[skip + i] = static_cast<uint16_t>(__float_as_uint(l[i]) >> 16);
    else
      held[skip + i] = l[i];
  }
  const void *logits = bf16 ? static_cast<const void *>(held16.get() + skip) : held.get() + skip;
  auto bias = array<float>(e);
  for (int i = 0; i < e; ++i) bias[i] = static_cast<float>(0.2 * normal());
  auto ids = array<int32_t>(n * k);
  auto weights = array<float>(n * k), scores = array<float>(n * e);
  launch_route(c.p, c.r, logits, c.bias ? bias.get() : nullptr, ids.get(), c.weights ? weights.get() : nullptr,
               c.scores ? scores.get() : nullptr, nullptr);
  auto dw = array<float>(n * k), ds = array<float>(n * e), dl = array<float>(skip + n * e);
  auto dl16 = array<uint16_t>(skip + n * e);
  for (int i = 0; i < n * k; ++i) dw[i] = static_cast<float>(normal());
  for (int i = 0; i < n * e; ++i) ds[i] = static_cast<float>(normal());
  void *out = bf16 ? static_cast<void *>(dl16.get() + skip) : dl.get() + skip;
  launch_route_backward(c.p, c.r, logits, ids.get(), dw.get(), c.scores ? ds.get() : nullptr, out, nullptr);
  for (int t = 0; t < n; ++t) {
    const float *row = l.get() + t * e;
    const Token x = token(row, e, sigmoid);
    const std::vector<int> want = choices(c, row, c.bias ? bias.get() : nullptr, x);
    double sum = 0;
    for (int j = 0; j < k; ++j) {
      if (ids[t * k + j] != want[j]) emu::fail("a wrong choice");
      if (want[j] >= 0) sum += x.s[want[j]];
    }
    // (arguments of exponentials up to 120 apart)
    const double step = (400 + 2 * e) * 0x1p-23;
    std::vector<double> d(e), direct(e), m(e), m_direct(e);
    if (c.scores)
      for (int i = 0; i < e; ++i) {
        close(scores[t * e + i], x.s[i], step * x.s[i] + 0x1p-125, "score");
        d[i] = ds[t * e + i];
        m[i] = std::abs(d[i]);
      }
    double dot = 0, m_dot = 0;
    auto w_of = [&](int j) { return want[j] < 0 ? 0 : c.r.renormalize ? (sum > 0 ? x.s[want[j]] / sum : 0) : x.s[want[j]]; };
    for (int j = 0; j < k; ++j) {
      // (scores that all but vanish: renormalised over their own sum, in the kernel from their logits)
      if (c.weights && (sum > 1e-25 || !c.r.renormalize)) close(weights[t * k + j], w_of(j) * c.r.scale, step * w_of(j) * c.r.scale + 0x1p-100, "weight");
      const double u = want[j] < 0 ? 0 : dw[t * k + j] * static_cast<double>(c.r.scale);
      dot += u * w_of(j);
      m_dot += std::abs(u) * w_of(j);
    }
    if (c.r.renormalize && sum <= 1e-25) continue;
    for (int j = 0; j < k; ++j) {
      if (want[j] < 0) continue;
      const double u = dw[t * k + j] * static_cast<double>(c.r.scale), w = w_of(j);
      if (c.r.renormalize) {
        const double slope = sigmoid ? x.away[want[j]] : 1;
        direct[want[j]] += w * (u - dot) * slope;
        m_direct[want[j]] += w * (std::abs(u) + m_dot) * slope;
      } else {
        d[want[j]] += u;
        m[want[j]] += std::abs(u);
      }
    }
    dot = m_dot = 0;
    for (int i = 0; i < e && !sigmoid; ++i) dot += d[i] * x.s[i], m_dot += m[i] * x.s[i];
    for (int i = 0; i < e; ++i) {
      const double slope = sigmoid ? x.s[i] * x.away[i] : x.s[i];
      const double g = direct[i] + slope * (d[i] - dot), mag = m_direct[i] + slope * (m[i] + m_dot);
      const double got = bf16 ? __uint_as_float(static_cast<uint32_t>(dl16[skip + t * e + i]) << 16) : dl[skip + t * e + i];
      close(got, g, step * mag + (bf16 ? 0x1p-8 * (std::abs(g) + step * mag) : 0) + 1e-37, "gradient");
    }
  }
}

void quantize(int64_t blocks) {
  printf("quantize %lld blocks\n", static_cast<long long>(blocks));
  fflush(stdout);
  std::unique_ptr<uint16_t, void (*)(void *)> x(static_cast<uint16_t *>(aligned_alloc(16, blocks * 64)), free);
  std::unique_ptr<uint8_t, void (*)(void *)> codes(static_cast<uint8_t *>(aligned_alloc(16, blocks * 16)), free);
  auto scales = array<uint8_t>(blocks);
  for (int64_t i = 0; i < blocks * 32; ++i) x.get()[i] = static_cast<uint16_t>(f32_to_bf16(static_cast<float>(normal())));
  launch_quantize_mxfp4(blocks * 32, x.get(), codes.get(), scales.get(), nullptr);
  for (int64_t b = 0; b < blocks; ++b) {
    double top = 0;
    auto value = [&](int i) { return static_cast<double>(__uint_as_float(static_cast<uint32_t>(x.get()[b * 32 + i]) << 16)); };
    for (int i = 0; i < 32; ++i) top = std::max(top, std::abs(value(i)));
    const int e = top > 0 ? std::max(std::ilogb(top) - 2, -127) : -127;
    if (scales[b] != e + 127) emu::fail("a wrong scale");
    for (int i = 0; i < 32; ++i) {
      const uint32_t code = codes.get()[b * 16 + i / 2] >> 4 * (i % 2) & 15;
      if (code != emu::to_e2m1(static_cast<float>(std::ldexp(value(i), -e)))) emu::fail("a wrong code");
    }
  }
}

}  // namespace
}  // namespace moe

int main(int, char **argv) {
  const int seed = atoi(argv[1]), n = atoi(argv[2]);
  moe::draw.seed(seed);
  emu::rng.seed(seed);
  for (int64_t blocks : {1, 3, 31, 256, 257, 700}) moe::quantize(blocks);
  for (int i = 0; i < n; ++i) moe::one(moe::any());
  printf("no failures\n");
  fflush(stdout);
}
