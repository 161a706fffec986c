// Every form of the products with MX-FP4 weights, lane by lane on the CPU, over random sizes: every
// load and store inside its memory, every barrier met, no stage of LDS read before it
// has landed or freed while it is read, and the results right.
//
// GATED: the gated block, or the linear layer.  Arguments: seed, cases of each form.
#include "expert_mx.inc"

#include <sys/mman.h>

#include <memory>

namespace moe {
namespace {

std::mt19937 draw(1);
int upto(int n) { return static_cast<int>(draw() % n); }

// Memory of exactly n bytes, `align`-aligned and not more, that ends where it ends.
struct Bytes {
  std::unique_ptr<char[]> all;
  char *p;
  size_t n;
  // round: readable to the end of such a unit
  Bytes(size_t bytes, size_t align, bool written, size_t round = 1) : n(bytes) {
    const size_t whole = (bytes + round - 1) / round * round;
    all.reset(new char[align + whole]);  // (of 16 bytes' alignment)
    p = all.get() + align;
    emu::own(p, whole, written);
    memset(p, 0x7F, whole);
  }
};

struct Case {
  int experts, k, n, act, pad;
  bool bias, residual, codes;
  std::vector<int> counts;
};

double value4(const char *codes, int i) { return emu::e2m1(static_cast<uint8_t>(codes[i / 2]) >> 4 * (i % 2) & 15); }

double activation(int act, double z) {
  switch (act) {
    case MOE_ACT_SILU: return z / (1 + std::exp(-z));
    case MOE_ACT_GELU_TANH: return 0.5 * z * (1 + std::tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)));
    case MOE_ACT_RELU: return z < 0 ? 0 : z;
    default: return z;
  }
}

template <class S, bool GLU>
void one(const Case &c, const char *name) {
  emu::ranges.clear();
  const int k = c.k, wrows = GLU ? 2 * c.n : c.n, blocks = k / 32;
  const int x_bytes = S::FP8 ? k : k / 2, xs_bytes = S::FP8 ? k / 128 * 4 : blocks;
  std::vector<int32_t> offsets(c.experts + 1), counts(c.counts.begin(), c.counts.end());
  int64_t pairs = 0;
  for (int e = 0; e < c.experts; ++e) {
    offsets[e + 1] = offsets[e] + (counts[e] + c.pad - 1) / c.pad * c.pad;
    pairs += counts[e];
  }
  const int rows = offsets[c.experts];
  Bytes x(static_cast<size_t>(rows) * x_bytes, 16, false), xs(static_cast<size_t>(rows) * xs_bytes, 4, false, 4);
  Bytes w(static_cast<size_t>(c.experts) * wrows * (k / 2), 16, false);
  Bytes ws(static_cast<size_t>(c.experts) * wrows * blocks, 4, false, 4);
  Bytes y(static_cast<size_t>(rows) * c.n * (c.codes ? 1 : 4) / 2, 16, true);
  Bytes ys(c.codes ? static_cast<size_t>(rows) * (c.n / 32) : 0, 1, true);
  Bytes residual(c.residual ? static_cast<size_t>(rows) * c.n * 2 : 0, 16, false);
  std::vector<float> bias(c.bias ? c.experts * wrows : 0);
  for (float &b : bias) b = upto(9) * 0.25f - 1;
  for (size_t i = 0; i < w.n; ++i) w.p[i] = static_cast<char>(draw());
  for (size_t i = 0; i < ws.n; ++i) ws.p[i] = static_cast<char>(124 + upto(5));
  for (int e = 0; e < c.experts; ++e)  // rows without a token stay NaN
    for (int r = offsets[e]; r < offsets[e] + counts[e]; ++r) {
      for (int i = 0; i < x_bytes; ++i) {
        const int v = static_cast<int>(draw() & 255);
        x.p[static_cast<size_t>(r) * x_bytes + i] = static_cast<char>(S::FP8 ? (v & 0xB7) : v);  // below 2^1
      }
      for (int i = 0; i < (S::FP8 ? k / 128 : blocks); ++i) {
        const float f = std::ldexp(1.0f, upto(4) - 2);
        if (S::FP8)
          memcpy(xs.p + static_cast<size_t>(r) * xs_bytes + i * 4, &f, 4);
        else
          xs.p[static_cast<size_t>(r) * xs_bytes + i] = static_cast<char>(125 + upto(4));
      }
      for (int i = 0; c.residual && i < c.n; ++i) {
        const uint16_t b = static_cast<uint16_t>(f32_to_bf16(upto(17) * 0.5f - 4));
        memcpy(residual.p + (static_cast<size_t>(r) * c.n + i) * 2, &b, 2);
      }
    }
  MxArgs g;
  g.x = x.p, g.x_scales = xs.p, g.w = w.p, g.w_scales = ws.p;
  g.bias = c.bias ? bias.data() : nullptr;
  g.residual = c.residual ? reinterpret_cast<uint16_t *>(residual.p) : nullptr;
  g.y = c.codes ? nullptr : reinterpret_cast<uint16_t *>(y.p);
  g.codes = c.codes ? reinterpret_cast<uint8_t *>(y.p) : nullptr;
  g.scales = c.codes ? reinterpret_cast<uint8_t *>(ys.p) : nullptr;
  g.offsets = offsets.data(), g.counts = counts.data();
  g.n_experts = c.experts, g.rows = rows, g.k = k, g.n = c.n, g.act = c.act;
  printf("%s experts %d rows %d K %d N %d pad %d bias %d residual %d codes %d\n", name, c.experts, rows, k, c.n, c.pad,
         c.bias, c.residual, c.codes);
  fflush(stdout);
  if (pairs == 0) return;
  // of a card of 8 and 16 units, so that workgroups take several tiles
  if (launch<S, GLU>(g, pairs, nullptr, S::kResident) != hipSuccess) emu::fail("launch");
  std::vector<double> z(wrows), mag(wrows), xv(k);
  for (int e = 0; e < c.experts; ++e)
    for (int r = offsets[e]; r < offsets[e + 1]; ++r) {
      const char *row = y.p + static_cast<size_t>(r) * c.n * (c.codes ? 1 : 4) / 2;
      if (r >= offsets[e] + counts[e]) {
        for (int i = 0; i < c.n * (c.codes ? 1 : 4) / 2; ++i)
          if (row[i] != 0x7F) emu::fail("a row without a token was written");
        continue;
      }
      if (rows > 64 && upto(16)) continue;  // some of many
      const char *xr = x.p + static_cast<size_t>(r) * x_bytes, *xsr = xs.p + static_cast<size_t>(r) * xs_bytes;
      for (int i = 0; i < k; ++i) {
        if (S::FP8) {
          float f;
          memcpy(&f, xsr + i / 128 * 4, 4);
          xv[i] = emu::e4m3(static_cast<uint8_t>(xr[i])) * f;
        } else {
          xv[i] = value4(xr, i) * emu::e8m0(static_cast<uint8_t>(xsr[i / 32]));
        }
      }
      for (int j = 0; j < wrows; ++j) {
        const size_t wr = static_cast<size_t>(e) * wrows + j;
        z[j] = c.bias ? bias[wr] : 0;
        mag[j] = std::abs(z[j]);
        for (int i = 0; i < k; ++i) {
          const double v = xv[i] * value4(w.p + wr * (k / 2), i) * emu::e8m0(static_cast<uint8_t>(ws.p[wr * blocks + i / 32]));
          z[j] += v;
          mag[j] += std::abs(v);
        }
      }
      for (int j = 0; j < c.n; ++j) {
        double want = activation(c.act, z[j]), far = (mag[j] * 2 + 1) * (k + 64) * 0x1p-23;
        if (GLU) {
          far = far * (std::abs(z[c.n + j]) + 1) + (std::abs(want) + mag[j]) * (mag[c.n + j] + 1) * (k + 64) * 0x1p-23;
          want *= z[c.n + j];
        }
        double got;
        if (c.codes) {
          const double unit = emu::e8m0(static_cast<uint8_t>(ys.p[static_cast<size_t>(r) * (c.n / 32) + j / 32]));
          got = value4(row, j) * unit;
          far += unit;  // half of the widest step; from 6 to the next power of two another 2
          if (std::abs(want) > 6 * unit) far += unit;
        } else {
          uint16_t b, add = 0;
          memcpy(&b, row + j * 2, 2);
          got = __uint_as_float(static_cast<uint32_t>(b) << 16);
          if (c.residual) memcpy(&add, residual.p + (static_cast<size_t>(r) * c.n + j) * 2, 2);
          want += __uint_as_float(static_cast<uint32_t>(add) << 16);
          far += (std::abs(want) + far) * 0x1p-8;
        }
        if (!(std::abs(got - want) <= far)) {
          fprintf(stderr, "row %d column %d: %g, wanted %g, may be off by %g\n", r, j, got, want, far);
          emu::fail("a wrong result");
        }
      }
    }
}

template <class S, bool GLU>
void some(int times, const char *name) {
  for (int i = 0; i < times; ++i) {
    emu::landing = static_cast<emu::Landing>(upto(3));
    Case c;
    c.experts = 1 + upto(upto(4) ? 3 : 70);
    const int unit = S::FP8 ? 128 : S::ODD ? 32 : 128;
    c.k = unit * (1 + upto(upto(3) ? 900 / unit : S::BI <= 16 ? 4500 / unit : 1800 / unit));
    if (S::ODD && c.k % 128 == 0) c.k += 32 * (1 + upto(3));
    c.n = 8 * (1 + upto(upto(3) ? 9 : 45));
    c.pad = upto(2) ? 1 : 1 + upto(40);
    c.act = upto(4);
    c.bias = upto(2);
    c.residual = !GLU && upto(2);
    c.codes = GLU && upto(2);
    if (c.codes) c.n = (c.n + 31) / 32 * 32;
    c.counts.resize(c.experts);
    int left = 20 + upto(S::BI * 5);
    for (int &n : c.counts) left -= n = upto(4) ? upto(std::min(left, S::BI * 2 + 3) + 1) : 0;
    one<S, GLU>(c, name);
  }
}

// Zeros that take no memory until they are written, between pages that cannot be touched.
struct Far {
  char *all, *p;
  size_t n;
  Far(size_t bytes, size_t align, bool written, size_t round = 1) {
    const size_t whole = (bytes + round - 1) / round * round, pages = (whole + align + 4095) / 4096 * 4096;
    n = pages + 8192;
    all = static_cast<char *>(mmap(nullptr, n, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
    if (all == MAP_FAILED || mprotect(all + 4096, pages, PROT_READ | PROT_WRITE)) emu::fail("mmap");
    p = all + 4096 + (pages - whole) / align * align;
    emu::own(p, whole, written);
  }
  ~Far() { munmap(all, n); }
};

// The largest layers and buffers: addresses alone, without products.  kFarWork: rows of operands
// that the tiles of a case load in all their steps.
constexpr int64_t kFarWork = 600000;
template <class S, bool GLU>
void far_away(int times, const char *name) {
  emu::no_products = true;
  for (int i = 0; i < times; ++i) {
    emu::ranges.clear();
    emu::landing = static_cast<emu::Landing>(upto(3));
    const int unit = S::FP8 ? 128 : S::ODD ? 32 : 128, most = 1 << (11 + upto(10));
    int k = unit * (1 + upto(most / unit));
    if (S::ODD && k % 128 == 0) k -= 32;
    int n = 8 * (1 + upto(1 << 17));
    const bool codes = GLU && upto(2), residual = !GLU && upto(2);
    if (codes) n = (n + 31) / 32 * 32;
    if (upto(4) == 0) n = 8 * (1 + upto(20)) / (codes ? 4 : 1) * (codes ? 4 : 1);
    if (codes) n = std::max(n / 32 * 32, 32);
    while (static_cast<int64_t>(k) * n >= int64_t{1} << 29) n = std::max(n / 64 * 32, 32);
    const int experts = 1 + upto(upto(2) ? 4 : 1024), wrows = GLU ? 2 * n : n;
    // few rows of some experts, anywhere in the buffer
    std::vector<int32_t> offsets(experts + 1), counts(experts);
    // (2^45 bytes at most: what a process can name)
    const int64_t last = std::min<int64_t>(2147000000, (int64_t{1} << 44) / std::max(k, 2 * n)) - 2000000;
    int64_t pairs = 0, at = 0;
    for (int e = 0; e < experts; ++e) {
      offsets[e] = static_cast<int32_t>(at);
      if (upto(experts) < 2 && pairs < 3 * S::BI) counts[e] = 1 + upto(S::BI + 2);
      pairs += counts[e];
      at = std::min<int64_t>(at + counts[e] + draw() % (2 * last / experts), last + 1000 * e);
    }
    if (pairs == 0) counts[0] = 1, pairs = 1;
    for (int e = 0; e + 1 < experts; ++e) offsets[e + 1] = std::max(offsets[e + 1], offsets[e] + counts[e]);
    const int rows = offsets[experts] = offsets[experts - 1] + counts[experts - 1];
    const int64_t x_bytes = S::FP8 ? k : k / 2, xs_bytes = S::FP8 ? k / 128 * 4 : k / 32;
    // what is left of a tile's steps and columns after a while tells nothing new
    const int64_t col_tiles = (n + S::BJ / (GLU ? 2 : 1) - 1) / (S::BJ / (GLU ? 2 : 1));
    if ((pairs / S::BI + 3) * col_tiles * (k / 256 + 1) * (S::BI + S::BJ) > kFarWork) {
      --i;
      continue;
    }
    printf("%s far: experts %d rows %d of %lld K %d N %d residual %d codes %d\n", name, experts, rows,
           static_cast<long long>(pairs), k, n, residual, codes);
    fflush(stdout);
    Far x(rows * x_bytes, 16, false), xs(rows * xs_bytes, 4, false, 4);
    Far w(static_cast<size_t>(experts) * wrows * (k / 2), 16, false);
    Far ws(static_cast<size_t>(experts) * wrows * (k / 32), 4, false, 4);
    Far y(static_cast<size_t>(rows) * n * (codes ? 1 : 4) / 2, 16, true);
    Far ys(codes ? static_cast<size_t>(rows) * (n / 32) : 16, 1, true);
    Far add(residual ? static_cast<size_t>(rows) * n * 2 : 16, 16, false);
    Far bias(static_cast<size_t>(experts) * wrows * 4, 16, false);
    MxArgs g;
    g.x = x.p, g.x_scales = xs.p, g.w = w.p, g.w_scales = ws.p;
    g.bias = reinterpret_cast<float *>(bias.p);
    g.residual = residual ? reinterpret_cast<uint16_t *>(add.p) : nullptr;
    g.y = codes ? nullptr : reinterpret_cast<uint16_t *>(y.p);
    g.codes = codes ? reinterpret_cast<uint8_t *>(y.p) : nullptr;
    g.scales = codes ? reinterpret_cast<uint8_t *>(ys.p) : nullptr;
    g.offsets = offsets.data(), g.counts = counts.data();
    g.n_experts = experts, g.rows = rows, g.k = k, g.n = n, g.act = upto(4);
    if (launch<S, GLU>(g, pairs, nullptr, S::kResident) != hipSuccess) emu::fail("launch");
  }
  emu::no_products = false;
}

template <class S, bool GLU>
void all(int n, const char *name) {
  some<S, GLU>(n, name);
  far_away<S, GLU>(n / 4, name);
}

template <bool GLU>
void forms(int n) {
  // launch_sized's
  all<MxShape<16, 64, 1, 1, 3, false, false, true, 4>, GLU>(n, "16x64, K in four");
  all<MxShape<16, 64, 1, 1, 3, false, true, true, 4>, GLU>(n, "16x64, K in four, odd");
  all<MxShape<16, 64, 1, 1, 2, true, false, true, 4>, GLU>(n, "16x64, K in four, FP8");
  all<MxShape<16, 64, 1, 1, 2, false, false, true>, GLU>(n, "16x64");
  all<MxShape<16, 64, 1, 1, 2, false, true, true>, GLU>(n, "16x64, odd");
  all<MxShape<16, 64, 1, 1, 2, true, false, true>, GLU>(n, "16x64, FP8");
  all<MxShape<128, 128, 2, 2, 2, false, false, false>, GLU>(n, "128x128");
  all<MxShape<128, 128, 2, 2, 2, false, true, false>, GLU>(n, "128x128, odd");
  all<MxShape<64, 128, 4, 1, 2, true, false, false>, GLU>(n, "64x128, FP8");
  all<MxShape<128, 256, 4, 2, 2, true, false, false>, GLU>(n, "128x256, FP8");
  all<MxShape<256, 256, 2, 4, 2, false, false, false>, GLU>(n, "256x256");
}

}  // namespace
}  // namespace moe

int main(int, char **argv) {
  const int seed = atoi(argv[1]), n = atoi(argv[2]);
  moe::draw.seed(seed);
  emu::rng.seed(seed);
  moe::forms<GATED>(n);
  printf("no failures\n");
  fflush(stdout);
}
