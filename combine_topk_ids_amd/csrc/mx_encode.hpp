// mx_encode.hpp -- MX-FP4 encoding of values that four lanes hold, eight to a lane.
#pragma once

#include "moe_device.hpp"

namespace moe {

constexpr uint32_t kMxNaN = 255;  // E8M0's NaN

// Magnitude bits of the largest of a lane's eight values (an infinity's or a NaN's above all).
__device__ __forceinline__ uint32_t mx_lane_max(const float (&v)[8]) {
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return am;
}

// The lane's eight codes (value i in bits 4i..4i+3) and the scale byte of its block, whose
// largest magnitude has bits `am`.  A block with an infinity or a NaN has the NaN scale and
// zero codes.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8], uint32_t am, uint32_t &scale) {
  const int x = mx_exponent(am);
  const float mul = __uint_as_float(static_cast<uint32_t>(127 - x) << 23);  // 2^-X
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * mul;
  // (the conversion saturates a NaN; such a block's codes are dropped)
  const uint32_t c = e2m1_lane8(q, true);
  const bool bad = am >= 0x7F800000u;
  scale = bad ? kMxNaN : static_cast<uint32_t>(x + 127);
  return bad ? 0u : c;
}

}  // namespace moe
