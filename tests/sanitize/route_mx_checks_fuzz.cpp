// Fuzz driver for the host-side rules of routing, quantisation and the products with MX-FP4
// weights (host_checks.cpp), built with address and undefined-behaviour sanitizers by
// tests/test_sanitizers_route_mx.py.  Besides the sanitizers' own checks it asserts what the
// kernels rely on for every router and layer that is accepted.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "host_checks.hpp"

namespace {

uint64_t state = 0x13198A2E03707344ull;
uint64_t next_u64() {  // splitmix64
  uint64_t z = (state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
template <typename T, size_t N>
T pick(const T (&v)[N]) { return v[next_u64() % N]; }

int failures = 0;
#define EXPECT(c)                                                                    \
  do {                                                                               \
    if (!(c) && failures++ < 20) fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c); \
  } while (0)

const int32_t kInt[] = {INT32_MIN, -1, 0, 1, 2, 3, 4, 8, 16, 32, 1024, INT32_MAX};
const int32_t kDim[] = {INT32_MIN, -32, 0, 1, 8, 32, 96, 128, 160, 4096, 16384, 32736, 32760, 1 << 20, (1 << 20) + 32, INT32_MAX};

int32_t small(int32_t n) { return next_u64() % 16 ? static_cast<int32_t>(1 + next_u64() % n) : pick(kInt); }
int32_t option(int32_t n) { return next_u64() % 16 ? static_cast<int32_t>(next_u64() % n) : pick(kInt); }
int32_t draw_dim() { return next_u64() % 2 ? pick(kDim) : static_cast<int32_t>(8 * (next_u64() % 4096)); }

moe_problem draw_problem() {
  moe_problem p = {};
  p.n_tokens = next_u64() % 8 ? static_cast<int64_t>(next_u64() % (1 << (next_u64() % 24))) : static_cast<int64_t>(next_u64());
  p.hidden = static_cast<int32_t>(8 * (1 + next_u64() % 1000));
  p.n_experts = 1 + static_cast<int32_t>(next_u64() % 1024);
  p.top_k = 1 + static_cast<int32_t>(next_u64() % 8);
  p.ep = 1;
  p.pad_multiple = 1 + static_cast<int32_t>(next_u64() % 128);
  return p;
}

}  // namespace

int main(int argc, char **argv) {
  const long n = argc > 1 ? atol(argv[1]) : 100000;
  const uintptr_t ptr[] = {0, 1 << 20, (1 << 20) + 16, (1 << 20) + 2};
  auto u8 = [&] { return reinterpret_cast<uint8_t *>(pick(ptr)); };
  auto u16 = [&] { return reinterpret_cast<uint16_t *>(pick(ptr)); };
  auto i32 = [&] { return reinterpret_cast<int32_t *>(pick(ptr)); };
  auto f32 = [&] { return reinterpret_cast<float *>(pick(ptr)); };
  long routers = 0, layers = 0;
  for (long i = 0; i < n; ++i) {
    const moe_problem p = draw_problem();
    const float scale[] = {1.0f, -2.5f, 0.0f, INFINITY, NAN};
    const moe_router r = {option(2), option(2), next_u64() % 2 ? 1 : small(p.n_experts), small(8), small(2),
                          option(2), next_u64() % 4 ? 1.0f : pick(scale)};
    int rc = moe::host::check_router(&p, &r);
    const int f = moe::host::check_route_args(&p, &r, u16(), f32(), i32(), f32(), f32());
    const int b = moe::host::check_route_backward_args(&p, &r, u16(), i32(), f32(), f32(), u16());
    EXPECT(rc == MOE_OK || rc == MOE_EINVAL || rc == MOE_EOVERFLOW);
    EXPECT(f <= 0 && b <= 0);
    if (rc == MOE_OK) {
      ++routers;
      EXPECT(p.n_experts % r.n_groups == 0 && r.top_groups >= 1 && r.top_groups <= r.n_groups);
      EXPECT(p.top_k <= r.top_groups * (p.n_experts / r.n_groups) && p.top_k <= 64 && p.n_experts <= 1024);
      EXPECT(isfinite(r.scale));
    } else {
      EXPECT(f == rc && b == rc);
    }
    const int64_t rows = next_u64() % 4 ? static_cast<int64_t>(next_u64() % (1 << 30)) : static_cast<int64_t>(next_u64());
    const int32_t cols = draw_dim();
    if (moe::host::check_quantize_args(rows, cols, u16(), u8(), u8()) == MOE_OK) {
      EXPECT(rows >= 0 && cols > 0 && cols % 32 == 0);
      EXPECT(rows <= (int64_t{1} << 46) / cols);  // rows * cols does not overflow
    }
    const moe_expert_op op = {draw_dim(), draw_dim(), option(4), next_u64() % 4 ? 1 + static_cast<int32_t>(next_u64() % 2) : pick(kInt)};
    rc = moe::host::check_expert_mx_op(&p, &op);
    EXPECT(rc == MOE_OK || rc == MOE_EINVAL || rc == MOE_EOVERFLOW);
    moe_plan plan = {};
    plan.expert_counts = i32();
    plan.expert_offsets = i32();
    const int a = moe::host::check_expert_mx_args(&p, &plan, &op, u16(), u8(), u8(), u8(), f32(), u16(), u16(), u8());
    EXPECT(a <= 0);
    if (rc != MOE_OK) {
      EXPECT(a == rc);
      continue;
    }
    ++layers;
    const int64_t in = op.in_dim, out = op.out_dim;
    EXPECT(in > 0 && out > 0 && in % 32 == 0 && out % 8 == 0);
    EXPECT(op.fmt == MOE_FMT_MXFP4_B32 || in % 128 == 0);
    EXPECT(2 * out * (in / 2) < (int64_t{1} << 31));     // an expert's weights, bytes
    EXPECT(256 * in < (int64_t{1} << 31));               // a tile's rows, bytes (FP8: 128 of them)
    EXPECT(256 * out * 2 < (int64_t{1} << 31));          // a tile's results, bytes
    EXPECT(2 * out * (in / 32) + 3 < (int64_t{1} << 31));  // an expert's scales, whole words
  }
  EXPECT(routers > n / 50);
  EXPECT(layers > n / 50);
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("no failures in %ld draws (%ld routers, %ld layers accepted)\n", n, routers, layers);
  return 0;
}
