// Fuzz driver for the experts' host-side rules (host_checks.cpp), built with
// address and undefined-behaviour sanitizers by tests/test_sanitizers_expert.py.
// Problems and layers are drawn from edge values of every field and from
// random ones; besides the sanitizers' own checks it asserts what the kernels
// rely on for every layer that check_expert_op accepts.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "host_checks.hpp"

namespace {

uint64_t state = 0x243F6A8885A308D3ull;
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

const int32_t kDim[] = {INT32_MIN, -8, 0, 1, 8, 64, 120, 128, 256, 1000, 4096, 16384, 32760, 32768, 1 << 20,
                        (1 << 20) + 8, INT32_MAX - 7, INT32_MAX};
const int32_t kEnum[] = {-1, 0, 1, 2, 3, 4, INT32_MAX};

moe_problem draw_problem() {
  moe_problem p;
  p.n_tokens = next_u64() % 8 ? static_cast<int64_t>(next_u64() % (1 << (next_u64() % 24))) : static_cast<int64_t>(next_u64());
  p.hidden = static_cast<int32_t>(8 * (1 + next_u64() % 1000));
  p.n_experts = 1 + static_cast<int32_t>(next_u64() % 1024);
  p.top_k = 1 + static_cast<int32_t>(next_u64() % 8);
  p.ep = 1;
  p.recv_capacity = 0;
  p.pad_multiple = 1 + static_cast<int32_t>(next_u64() % 128);
  p.fmt = 0;
  p.flags = 0;
  p.expert_capacity = 0;
  if (next_u64() % 4 == 0) {
    p.pad_multiple = 1;
    p.expert_capacity = 1 + static_cast<int64_t>(next_u64() % 5000);
  }
  return p;
}

int32_t draw_dim() { return next_u64() % 2 ? pick(kDim) : static_cast<int32_t>(8 * (next_u64() % 4096)); }

}  // namespace

int main(int argc, char **argv) {
  const long n = argc > 1 ? atol(argv[1]) : 100000;
  const uintptr_t ptr[] = {0, 1 << 20, (1 << 20) + 16, (1 << 20) + 2};
  long accepted = 0;
  for (long i = 0; i < n; ++i) {
    const moe_problem p = draw_problem();
    moe_expert_op op = {draw_dim(), draw_dim(), next_u64() % 4 ? static_cast<int32_t>(next_u64() % 4) : pick(kEnum),
                        next_u64() % 4 ? static_cast<int32_t>(next_u64() % 2) : pick(kEnum)};
    const int rc = moe::host::check_expert_op(&p, &op);
    EXPECT(rc == MOE_OK || rc == MOE_EINVAL || rc == MOE_EOVERFLOW);
    moe_plan plan = {};
    plan.expert_counts = reinterpret_cast<int32_t *>(pick(ptr));
    plan.expert_offsets = reinterpret_cast<int32_t *>(pick(ptr));
    plan.slot = reinterpret_cast<int32_t *>(pick(ptr));
    auto u16 = [&] { return reinterpret_cast<uint16_t *>(pick(ptr)); };
    auto f32 = [&] { return reinterpret_cast<float *>(pick(ptr)); };
    const int f = moe::host::check_expert_forward_args(&p, &plan, &op, u16(), f32(), u16(), f32(), f32(), u16(),
                                                       u16(), u16());
    const int b = moe::host::check_expert_backward_args(&p, &plan, &op, next_u64() % 2, u16(), u16(), u16(), u16(),
                                                        u16(), u16(), u16(), f32(), u16());
    const int c = moe::host::check_combine_backward_args(&p, &plan, u16(), f32(), u16(), u16(), f32());
    EXPECT(f <= 0 && b <= 0 && c <= 0);
    if (rc != MOE_OK) {
      EXPECT(f == rc && b == rc);
      continue;
    }
    ++accepted;
    const int64_t in = op.in_dim, out = op.out_dim, unit = op.fmt == MOE_FMT_BF16 ? 8 : 128;
    EXPECT(in > 0 && out > 0 && in % unit == 0 && out % unit == 0);
    EXPECT(2 * out * in * 2 < (int64_t{1} << 31));                 // an expert's weights, bytes
    EXPECT(256 * (in > 2 * out ? in : 2 * out) * 2 < (int64_t{1} << 31));  // a tile's rows, bytes
    const int64_t rows = moe::expert_row_bound(p);
    EXPECT(rows >= 0 && rows <= moe::max_rows(p) && rows <= p.n_tokens * p.top_k);
    // workgroups of 512 threads of a launch: below 2^32 threads
    const int64_t wide = (in > 2 * out ? in : 2 * out) / 64 + 1;
    EXPECT((rows / 64 + p.n_experts) * wide * 512 < (int64_t{1} << 32));
    EXPECT(moe::expert_workspace_bytes(p, op) % 256 == 0);
    EXPECT(moe::expert_workspace_bytes(p, op) >=
           static_cast<size_t>(moe::max_rows(p) / moe::kBiasChunkRows + p.n_experts) * 2 * out * 4);
  }
  EXPECT(accepted > n / 50);
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("no failures in %ld layers (%ld accepted)\n", n, accepted);
  return 0;
}
