// A wave of 64 lanes on the CPU: what the kernels name of HIP and of the compiler's builtins, so
// that their sources run under a host compiler, with every access checked.
//
// Each lane is a fiber; an operation across lanes meets the wave's 64 first (and ends the
// program if they come to different ones), a barrier the workgroup's.  Workgroups run one after
// another, the waves of one in an order drawn anew after every barrier.  Loads to LDS land late
// (when a wait asks for them), at once, or one or the other by chance (emu::landing): what reads a
// stage too early sees the poison or the tile before, what frees one too early loses it.  Loads and
// stores through a buffer resource must end in memory that emu::own() names; everything else is left to the
// address sanitizer.  What this cannot show is what a compiler makes of the sources for the GPU.
#pragma once
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <bit>
#include <cmath>
#include <deque>
#include <functional>
#include <map>
#include <random>
#include <string>
#include <type_traits>
#include <vector>

#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __launch_bounds__(...)

typedef void *hipStream_t;
typedef int hipError_t;
constexpr hipError_t hipSuccess = 0;
inline hipError_t hipGetLastError() { return hipSuccess; }

struct alignas(16) float4 { float x, y, z, w; };
struct alignas(8) float2 { float x, y; };
struct alignas(16) uint4 { uint32_t x, y, z, w; };
struct alignas(8) uint2 { uint32_t x, y; };
struct dim3 { uint32_t x = 1, y = 1, z = 1; };
inline dim3 threadIdx, blockIdx, blockDim, gridDim;

using std::max;
using std::min;

namespace emu {

[[noreturn]] inline void fail(const char *what) {
  fprintf(stderr, "workgroup %u, thread %u: %s\n", blockIdx.x, threadIdx.x, what);
  abort();
}

// ---- memory that buffer resources may reach -----------------------------------

struct Range {
  const char *from, *to;
  bool written;
};
inline std::vector<Range> ranges;
inline void own(const void *p, size_t bytes, bool written) {
  ranges.push_back({static_cast<const char *>(p), static_cast<const char *>(p) + bytes, written});
}
inline void touch(const char *p, size_t bytes, bool write) {
  for (const Range &r : ranges)
    if (p >= r.from && p + bytes <= r.to) {
      if (write && !r.written) fail("a store into an input");
      return;
    }
  fail(write ? "a store outside its memory" : "a load outside its memory");
}

// ---- fibers ----------------------------------------------------------------------

constexpr int kLanes = 64;
constexpr size_t kStack = 256 << 10;
enum class At { kReady, kLanes, kBarrier, kDone };
struct Load {
  const char *base;
  uint32_t records, off[kLanes];
  char *to;
  int bytes;  // of a lane; 0: a store
};
struct Wave {
  const void *args[kLanes];
  std::string kind;
  int arrived = 0;
  std::deque<Load> pending;
};
struct Fiber {
  void *sp = nullptr;
  At at = At::kDone;
};
inline std::vector<char *> stacks;
inline std::vector<Fiber> fibers;
inline std::vector<Wave> waves;
inline void *home;
inline int current;
inline std::function<void()> *body;
inline std::mt19937 rng(1);
enum Landing { kLate, kAtOnce, kEither };
inline Landing landing = kLate;
inline bool no_products = false;  // the matrix instruction leaves its sum as it is

// Saves what a call keeps, and changes stacks.
__attribute__((naked, noinline)) inline void change(void **, void *) {
  __asm__ __volatile__(
      "pushq %rbp\n\tpushq %rbx\n\tpushq %r12\n\tpushq %r13\n\tpushq %r14\n\tpushq %r15\n\t"
      "movq %rsp, (%rdi)\n\tmovq %rsi, %rsp\n\t"
      "popq %r15\n\tpopq %r14\n\tpopq %r13\n\tpopq %r12\n\tpopq %rbx\n\tpopq %rbp\n\tret");
}
inline void leave(At at) {
  fibers[current].at = at;
  change(&fibers[current].sp, home);
}
inline void begin() {
  (*body)();
  leave(At::kDone);
  abort();
}
inline int lane() { return current % kLanes; }
inline Wave &wave() { return waves[current / kLanes]; }

// f(the lanes' arguments) once, by the last lane to come.
template <class A, class F>
void together(const char *kind, const A &arg, F f) {
  Wave &w = wave();
  if (w.arrived == 0) w.kind = kind;
  if (w.kind != kind) fail(("lanes of a wave at different operations: " + w.kind + ", " + kind).c_str());
  w.args[lane()] = &arg;
  if (++w.arrived < kLanes) return leave(At::kLanes);
  const A *all[kLanes];
  for (int l = 0; l < kLanes; ++l) all[l] = static_cast<const A *>(w.args[l]);
  f(all);
  w.arrived = 0;
  const int first = current / kLanes * kLanes;
  for (int l = 0; l < kLanes; ++l)
    if (first + l != current) fibers[first + l].at = At::kReady;
}

inline void land(const Load &m) {
  for (int l = 0; l < kLanes; ++l)
    for (int d = 0; d < m.bytes; d += 4) {
      const uint64_t off = static_cast<uint64_t>(m.off[l]) + d;
      char *to = m.to + l * m.bytes + d;
      if (off + 4 <= m.records) {
        touch(m.base + off, 4, false);
        memcpy(to, m.base + off, 4);
      } else {
        memset(to, 0, 4);
      }
    }
}
inline void issued(const Load &m) {
  const bool now = m.bytes == 0 || landing == kAtOnce || (landing == kEither && rng() % 2);
  if (now && m.bytes) land(m);
  wave().pending.push_back(m);
  if (now) wave().pending.back().bytes = 0;
  if (wave().pending.size() > 4096) fail("loads that nothing waits for");
}
// at most n of the wave's loads and stores under way
inline void land_all_but(size_t n) {
  auto &q = wave().pending;
  for (; q.size() > n; q.pop_front())
    if (q.front().bytes) land(q.front());
}

inline void barrier() { leave(At::kBarrier); }

// A workgroup's LDS, poisoned.
inline std::map<std::string, std::vector<char>> shared_memory;
inline char *shared_bytes(const char *name, size_t bytes) {
  auto &m = shared_memory[name];
  if (m.empty()) m.assign(bytes, 0x7F);  // FP8's and bf16's NaN
  return m.data();
}
template <class T>
T *shared(const char *name, size_t n) {
  return reinterpret_cast<T *>(shared_bytes(name, n * sizeof(T)));
}

template <class F>
void launch(uint32_t grid, uint32_t threads, F kernel) {
  if (threads % kLanes) fail("a workgroup of no whole waves");
  if (grid == 0 || static_cast<uint64_t>(grid) * threads >> 32) fail("a grid that cannot be launched");
  std::function<void()> one = kernel;
  body = &one;
  gridDim.x = grid;
  blockDim.x = threads;
  while (stacks.size() < threads) stacks.push_back(static_cast<char *>(aligned_alloc(4096, kStack)));
  for (uint32_t b = 0; b < grid; ++b) {
    blockIdx.x = b;
    shared_memory.clear();
    const int n = static_cast<int>(threads), n_waves = n / kLanes;
    fibers.assign(n, Fiber());
    waves.assign(n_waves, Wave());
    for (int t = 0; t < n; ++t) {
      void **top = reinterpret_cast<void **>(stacks[t] + kStack - 64);
      *--top = nullptr;  // (a return address: the stack's alignment at a function's entry)
      *--top = reinterpret_cast<void *>(&begin);
      for (int r = 0; r < 6; ++r) *--top = nullptr;
      fibers[t] = {top, At::kReady};
    }
    std::vector<int> order(n_waves);
    for (int w = 0; w < n_waves; ++w) order[w] = w;
    for (;;) {
      std::shuffle(order.begin(), order.end(), rng);
      for (int w : order)
        for (bool more = true; more;) {
          more = false;
          for (int l = 0; l < kLanes; ++l) {
            const int t = w * kLanes + l;
            if (fibers[t].at != At::kReady) continue;
            more = true;
            current = t;
            threadIdx.x = t;
            change(&home, fibers[t].sp);
          }
        }
      int at[4] = {};
      for (const Fiber &f : fibers) ++at[static_cast<int>(f.at)];
      if (at[static_cast<int>(At::kDone)] == n) break;
      if (at[static_cast<int>(At::kBarrier)] != n) fail("some threads at a barrier, others not");
      for (Fiber &f : fibers) f.at = At::kReady;
    }
    for (Wave &w : waves)
      for (const Load &m : w.pending)
        if (m.bytes) fail("a workgroup ends with loads to its LDS under way");
  }
}

// ---- operations across lanes -----------------------------------------------------

template <class T>
struct Pair {
  T v;
  int from;
  T *out;
};
// v of the lane that each names
template <class T>
T value_of(const char *kind, T v, int from) {
  T out;
  together(kind, Pair<T>{v, from, &out}, [](auto &all) {
    for (int l = 0; l < kLanes; ++l) {
      if (all[l]->from < 0 || all[l]->from >= kLanes) fail("a lane that is none");
      *all[l]->out = all[all[l]->from]->v;
    }
  });
  return out;
}
struct Bool {
  bool v;
  uint64_t *out;
};
inline uint64_t ballot(bool v) {
  uint64_t out;
  together("ballot", Bool{v, &out}, [](auto &all) {
    uint64_t m = 0;
    for (int l = 0; l < kLanes; ++l) m |= static_cast<uint64_t>(all[l]->v) << l;
    for (int l = 0; l < kLanes; ++l) *all[l]->out = m;
  });
  return out;
}
inline void meet() {
  together("lanes meet", 0, [](auto &) {});
}
template <class T>
T first_lane(T v) {
  T out;
  together("readfirstlane", Pair<T>{v, 0, &out}, [](auto &all) {
    for (int l = 0; l < kLanes; ++l) {
      if (all[l]->v != all[0]->v) fail("readfirstlane of values that differ");
      *all[l]->out = all[0]->v;
    }
  });
  return out;
}

inline int dpp(int old, int v, int ctrl, int row_mask, int bank_mask, bool bound_zero) {
  const int l = lane(), row = l / 16, in = l % 16;
  int from = -1;
  if (ctrl < 0x100) from = l / 4 * 4 + (ctrl >> 2 * (l % 4) & 3);
  else if (ctrl > 0x110 && ctrl < 0x120) from = in >= ctrl - 0x110 ? l - (ctrl - 0x110) : -1;
  else if (ctrl == 0x140) from = row * 16 + 15 - in;
  else if (ctrl == 0x141) from = l / 8 * 8 + 7 - l % 8;
  else if (ctrl == 0x142) from = row > 0 ? row * 16 - 1 : -1;
  else if (ctrl == 0x143) from = l >= 32 ? 31 : -1;
  else fail("an unknown DPP control");
  const int got = value_of("dpp", v, from < 0 ? l : from);
  if (!(row_mask >> row & 1) || !(bank_mask >> (in / 4) & 1)) return old;
  return from < 0 ? (bound_zero ? 0 : old) : got;
}

struct Two {
  uint32_t v[2];
  uint32_t operator[](int i) const { return v[i]; }
  operator uint64_t() const = delete;
};
// rows of `run` lanes: odd ones of a change places with even ones of b
inline Two swap_rows(uint32_t a, uint32_t b, int run) {
  const int l = lane();
  const uint32_t a_other = value_of("swap", a, l ^ run), b_other = value_of("swap", b, l ^ run);
  return (l / run) % 2 ? Two{{b_other, b}} : Two{{a, a_other}};
}

// ---- buffers -------------------------------------------------------------------------

struct Resource {
  const char *base;
  uint32_t records;
};
template <class V>
V buffer_load(const Resource &r, int voffset, int soffset) {
  V v;
  uint32_t words[sizeof(V) / 4];
  for (size_t d = 0; d < sizeof(V) / 4; ++d) {
    const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(voffset)) + soffset + d * 4;
    words[d] = 0;
    if (off + 4 <= r.records) {
      touch(r.base + off, 4, false);
      memcpy(&words[d], r.base + off, 4);
    }
  }
  memcpy(&v, words, sizeof(V));
  return v;
}
template <class V>
void buffer_store(const V &v, const Resource &r, int voffset, int soffset) {
  const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(voffset)) + soffset;
  if (off + sizeof(V) <= r.records) {
    touch(r.base + off, sizeof(V), true);
    memcpy(const_cast<char *>(r.base) + off, &v, sizeof(V));
  }
  together("buffer store", 0, [](auto &) { issued(Load{}); });
}

template <int STRIDE, int BYTES, class R, int L>
void load_lds(const R &r, char *to, const uint32_t (&o)[L]) {
  struct Arg {
    uint32_t r[4];
    char *to;
    const uint32_t *o;
  } arg{{static_cast<uint32_t>(r[0]), static_cast<uint32_t>(r[1]), static_cast<uint32_t>(r[2]),
         static_cast<uint32_t>(r[3])},
        to, o};
  together("load to LDS", arg, [](auto &all) {
    for (int l = 1; l < kLanes; ++l)
      if (memcmp(all[l]->r, all[0]->r, 16) || all[l]->to != all[0]->to) fail("a load whose scalars differ");
    const uint64_t base = all[0]->r[0] | static_cast<uint64_t>(all[0]->r[1]) << 32;
    for (int u = 0; u < L; ++u) {
      Load m{reinterpret_cast<const char *>(base), all[0]->r[2], {}, all[0]->to + u * STRIDE, BYTES};
      for (int l = 0; l < kLanes; ++l) {
        m.off[l] = all[l]->o[u];
        if (m.off[l] < m.records && (base + m.off[l]) % 4) fail("a load that starts inside a word");
      }
      // (where it lands, whatever the landing: the sanitizer sees the whole of it)
      for (int i = 0; i < kLanes * BYTES; i += 4) {
        volatile uint32_t *p = reinterpret_cast<volatile uint32_t *>(m.to + i);
        *p = *p;
      }
      issued(m);
    }
  });
}
inline void wait_and_meet(int n) {
  together("wait", n, [](auto &all) { land_all_but(*all[0]); });
  barrier();
}

// ---- number formats and the matrix instruction -----------------------------------------

inline double e2m1(int c) {
  static const double v[8] = {0, .5, 1, 1.5, 2, 3, 4, 6};
  return c & 8 ? -v[c & 7] : v[c & 7];
}
inline double e4m3(int c) {
  const int e = c >> 3 & 15, m = c & 7;
  if (e == 15 && m == 7) return NAN;
  const double v = e ? std::ldexp(8 + m, e - 10) : std::ldexp(m, -9);
  return c & 128 ? -v : v;
}
inline double e8m0(int b) { return b == 255 ? NAN : std::ldexp(1.0, b - 127); }
inline uint32_t to_e2m1(float v) {
  const float a = std::fabs(v);
  const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
  return (a != a ? 7u : c) | (std::bit_cast<uint32_t>(v) >> 28 & 8u);
}
inline uint32_t pk_fp4(uint32_t old, float a, float b, int sel) {
  return (old & ~(0xFFu << 8 * sel)) | (to_e2m1(a) | to_e2m1(b) << 4) << 8 * sel;
}

// Value k of the 128 of lane-row r of an operand: 4 lane groups of 32.
template <class A, class B, class V>
V mfma_scaled(A a, B b, V c, int fmt_a, int fmt_b, int sel_a, int scale_a, int sel_b,
              int scale_b) {
  struct Arg {
    uint32_t x[2][8];
    int fmt[2], sel[2], scale[2];
    V c, *out;
  } arg{};
  V out;
  memcpy(arg.x[0], &a, fmt_a == 4 ? 16 : 32);
  memcpy(arg.x[1], &b, fmt_b == 4 ? 16 : 32);
  arg.fmt[0] = fmt_a, arg.fmt[1] = fmt_b, arg.sel[0] = sel_a, arg.sel[1] = sel_b;
  arg.scale[0] = scale_a, arg.scale[1] = scale_b;
  arg.c = c, arg.out = &out;
  if (no_products) return c;
  together("mfma", arg, [](auto &all) {
    static float v[2][16][128];
    for (int s = 0; s < 2; ++s)
      for (int l = 0; l < kLanes; ++l) {
        const auto &m = *all[l];
        const float scale = static_cast<float>(e8m0(m.scale[s] >> 8 * m.sel[s] & 255));
        const int r = l % 16, q = l / 16;
        for (int j = 0; j < 32; ++j) {
          if (m.fmt[s] == 4)
            v[s][r][32 * q + j] = static_cast<float>(e2m1(m.x[s][j / 8] >> 4 * (j % 8) & 15)) * scale;
          else
            v[s][r][j < 16 ? 16 * q + j : 64 + 16 * q + j - 16] =
                static_cast<float>(e4m3(m.x[s][j / 4] >> 8 * (j % 4) & 255)) * scale;
        }
      }
    for (int l = 0; l < kLanes; ++l)
      for (int i = 0; i < 4; ++i) {
        const float *x = v[0][l / 16 * 4 + i], *y = v[1][l % 16];
        float sum = 0;
        for (int k = 0; k < 128; ++k) sum += x[k] * y[k];
        (*all[l]->out)[i] = all[l]->c[i] + sum;
      }
  });
  return out;
}

}  // namespace emu

// ---- the names that the sources use ---------------------------------------------------------

typedef emu::Resource __amdgpu_buffer_rsrc_t;
#define __ballot(p) emu::ballot(p)
#define __builtin_amdgcn_readfirstlane(v) emu::first_lane(v)
#define __builtin_amdgcn_readlane(v, l) emu::value_of("readlane", static_cast<uint32_t>(v), l)
#define __builtin_amdgcn_mbcnt_lo(m, a) ((a) + __builtin_popcount((m) & static_cast<uint32_t>((1ull << std::min(emu::lane(), 32)) - 1)))
#define __builtin_amdgcn_mbcnt_hi(m, a) ((a) + __builtin_popcount((m) & static_cast<uint32_t>((1ull << std::max(emu::lane() - 32, 0)) - 1)))
#define __builtin_amdgcn_update_dpp(old, v, ctrl, row, bank, zero) emu::dpp(old, v, ctrl, row, bank, zero)
#define __builtin_amdgcn_permlane16_swap(a, b, fi, bc) emu::swap_rows(a, b, 16)
#define __builtin_amdgcn_permlane32_swap(a, b, fi, bc) emu::swap_rows(a, b, 32)
#define __builtin_amdgcn_fence(order, scope) ((void)0)
#define __builtin_amdgcn_wave_barrier() emu::meet()
#define __builtin_amdgcn_sched_group_barrier(a, b, c) ((void)0)
#define __builtin_amdgcn_sched_barrier(a) ((void)0)
#define __builtin_amdgcn_make_buffer_rsrc(p, stride, bytes, flags) \
  emu::Resource { static_cast<const char *>(static_cast<const void *>(p)), static_cast<uint32_t>(bytes) }
typedef uint32_t emu_u32x4 __attribute__((ext_vector_type(4)));
#define __builtin_amdgcn_raw_buffer_load_b128(r, v, s, policy) emu::buffer_load<emu_u32x4>(r, v, s)
#define __builtin_amdgcn_raw_buffer_store_b128(x, r, v, s, policy) emu::buffer_store(x, r, v, s)
#define __builtin_amdgcn_raw_buffer_store_b32(x, r, v, s, policy) emu::buffer_store(static_cast<uint32_t>(x), r, v, s)
#define __builtin_amdgcn_raw_buffer_store_b8(x, r, v, s, policy) emu::buffer_store(static_cast<uint8_t>(x), r, v, s)
#define __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4 emu::mfma_scaled
#define __builtin_amdgcn_alignbyte(hi, lo, n) \
  static_cast<uint32_t>(((static_cast<uint64_t>(hi) << 32) | (lo)) >> 8 * (n))
#define __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, sel) emu::pk_fp4(old, a, b, sel)
#define __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, sel) (emu::fail("not emulated"), 0)
#define __builtin_amdgcn_ds_read_tr16_b64_v4i16(p) (emu::fail("not emulated"), *(p))
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, x, y, z) (emu::fail("not emulated"), (c))
#define __builtin_amdgcn_exp2f(x) std::exp2(static_cast<float>(x))
#define __builtin_amdgcn_rcpf(x) (1.0f / static_cast<float>(x))
#define __expf(x) std::exp(static_cast<float>(x))
#define __syncthreads() emu::barrier()

inline uint32_t __float_as_uint(float f) { return std::bit_cast<uint32_t>(f); }
inline float __uint_as_float(uint32_t u) { return std::bit_cast<float>(u); }
inline int __shfl(int v, int from, int width = 64) {
  return emu::value_of("shfl", v, emu::lane() / width * width + (from & (width - 1)));
}
inline int __shfl_up(int v, int by, int width = 64) {
  const int l = emu::lane();
  return emu::value_of("shfl up", v, l % width >= by ? l - by : l);
}
inline float __shfl(float v, int from, int width = 64) {
  return std::bit_cast<float>(__shfl(std::bit_cast<int>(v), from, width));
}
