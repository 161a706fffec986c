// quantize.hip -- bf16 values to MX-FP4: per 32 values X = floor(log2 amax) - 2, scale byte
// X + 127, codes E2M1(x * 2^-X), rounded to nearest even and saturated.
//
// Bound by memory: 2 bytes read and 17/32 written a value.  Rows are whole blocks, so
// the array is one run of blocks; a lane holds 8 values, a quad a block.  131072 x 4096:
// 222 us, 6.1 TB/s.
#include "moe_device.hpp"
#include "moe_kernels.hpp"
#include "mx_encode.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;  // 16-byte pieces a thread reads

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__global__ __launch_bounds__(kThreads) void quantize_kernel(const uint16_t *x, uint8_t *codes, uint8_t *scales,
                                                            int64_t pieces) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads * kPieces;
  // (a block's four lanes are in or out together: pieces is a multiple of 4)
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads * kPieces + threadIdx.x;
       first - threadIdx.x < pieces; first += stride) {
    u32x4 raw[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int64_t at = first + u * kThreads;
      raw[u] = at < pieces ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x) + at)
                           : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int64_t at = first + u * kThreads;
      uint4 r4{raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      float v[8];
      unpack8(r4, v);
      uint32_t scale;
      const uint32_t c = mx_encode8(v, quad_max(mx_lane_max(v)), scale);
      if (at < pieces) {
        reinterpret_cast<uint32_t *>(codes)[at] = c;
        if ((threadIdx.x & 3) == 0) scales[at / 4] = static_cast<uint8_t>(scale);
      }
    }
  }
}

}  // namespace

hipError_t launch_quantize_mxfp4(int64_t values, const uint16_t *x, uint8_t *codes, uint8_t *scales,
                                 hipStream_t stream) {
  if (values == 0) return hipSuccess;
  const int64_t pieces = values / 8, per = kThreads * kPieces, blocks = (pieces + per - 1) / per;
  const uint32_t grid = static_cast<uint32_t>(blocks < (1 << 20) ? blocks : 1 << 20);
  quantize_kernel<<<grid, kThreads, 0, stream>>>(x, codes, scales, pieces);
  return hipGetLastError();
}

}  // namespace moe
