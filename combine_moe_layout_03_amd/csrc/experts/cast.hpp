// The cast of computed (float) channels to E4M3 codes with a scale per 128
// channels, as the FP8 dispatch casts bf16 rows: a lane holds 8 channels, a
// 16-lane DPP row a group.
#pragma once

#include "experts.hpp"

namespace moe {

constexpr uint32_t kInfBits = 0x7f800000u, kNanBits = 0x7fc00000u;

__device__ __forceinline__ float keep_finite(float h) {
  return __builtin_amdgcn_fmed3f(h, -3.402823466e38f, 3.402823466e38f);
}

// The bits of the largest |h|, of a NaN if there is one.
__device__ __forceinline__ uint32_t largest(const float (&h)[8]) {
  float m = fabsf(h[0]);
#pragma unroll
  for (int d = 1; d < 8; ++d) m = __builtin_elementwise_maximum(m, fabsf(h[d]));
  return __float_as_uint(m) & 0x7fffffffu;
}

// The scale of a group whose largest |h| has the bits `top`; NaN where spoilt.
template <int kFlags>
__device__ __forceinline__ float group_scale(uint32_t top, bool spoilt) {
  float am = __uint_as_float(top);
  if (am < 1e-4f) am = 1e-4f;
  // am / 448, correctly rounded (product, remainder, correction)
  const float s0 = am * (1.0f / 448.0f);
  float s = __builtin_fmaf(__builtin_fmaf(-448.0f, s0, am), 1.0f / 448.0f, s0);
  if (kFlags & kFp8RoundScale) {
    uint32_t b = __float_as_uint(s);
    if (b & 0x7fffffu) b = (b & 0xff800000u) + 0x800000u;
    s = __uint_as_float(b);
  }
  return spoilt ? __uint_as_float(kNanBits) : s;
}

// Codes of the correctly rounded h / s, as the cast of bf16 rows divides (none
// passes 448 by more than half a float step, which rounds to 448). One
// correction makes the reciprocal the correctly rounded one for every float
// significand (all 2^23 compared with 1 / s at six exponents).
__device__ __forceinline__ ex_u32x2 group_codes(const float (&h)[8], float s) {
  const float r = __builtin_amdgcn_rcpf(s), y = __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
  float d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = div_by_scale(h[i], s, y);
  return ex_u32x2{e4m3x4(d[0], d[1], d[2], d[3]), e4m3x4(d[4], d[5], d[6], d[7])};
}

}  // namespace moe
