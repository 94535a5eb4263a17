// What the routers share: reading a token's logits, their keys, the scores.
#pragma once

#include "experts.hpp"

namespace moe {

constexpr uint32_t kKeyNegInf = 0x007fffffu;  // the keys of the infinities
constexpr uint32_t kKeyPosInf = 0xff800000u;

__device__ __forceinline__ float gate_load(const void *x, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(x)[i] << 16)
              : static_cast<const float *>(x)[i];
}
// A token's logits lane + 64 j, all loads in flight together (past the last
// expert the last one's again, which the callers leave out).
template <int V>
__device__ __forceinline__ void gate_row(const void *x, int64_t row, int E, bool bf16,
                                         float (&v)[V]) {
  const int lane = threadIdx.x & 63;
  if (bf16) {
    const uint16_t *p = static_cast<const uint16_t *>(x) + row;
#pragma unroll
    for (int j = 0; j < V; ++j)
      v[j] = __uint_as_float((uint32_t)p[min(lane + 64 * j, E - 1)] << 16);
  } else {
    const float *p = static_cast<const float *>(x) + row;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = p[min(lane + 64 * j, E - 1)];
  }
}

// Key of a selectable logit, 0 for -infinity; NaN and +infinity also give 0 and
// set bad. The keys of the finite floats are those between the infinities',
// which NaN of either sign fall outside of.
__device__ __forceinline__ uint32_t gate_key(float x, bool *bad) {
  const int32_t u = (int32_t)__float_as_uint(x + 0.0f);
  const uint32_t k = (uint32_t)(u ^ ((u >> 31) | (int32_t)0x80000000));
  const bool fin = k - (kKeyNegInf + 1u) < kKeyPosInf - (kKeyNegInf + 1u);
  *bad = *bad || (!fin && k != kKeyNegInf);
  return fin ? k : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {  // 0 -> -infinity
  const int32_t u = (int32_t)k;
  const float f = __uint_as_float((uint32_t)(u ^ (~(u >> 31) | (int32_t)0x80000000)));
  return k ? f : -INFINITY;
}

// exp(d) for d <= 0: the exponent d log2(e) is rounded once, so the result is off
// by 2^-24 |d| and one step. Only for a sum over all experts, where the terms of
// large |d| are small against the first, which is 1; the gradient, where a term
// is an expert's own result, takes expf.
__device__ __forceinline__ float exp_below(float d) {
  return __builtin_amdgcn_exp2f(d * 1.44269504f);
}

__device__ __forceinline__ float log_sigmoid(float x) {  // x may be -infinity
  return fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// The scores of lanes 0 .. K-1 (x = the lane's logit, -infinity where there is
// none); top and sum are the softmax statistics over all experts.
template <int kMode>
__device__ __forceinline__ float gate_score(float x, float top, float sum) {
  constexpr bool kSig = kMode & kGateSigmoid, kRenorm = kMode & kGateRenorm;
  float p;
  if (kRenorm) {
    const float z = kSig ? log_sigmoid(x) : x;
    // the largest term of the selected ones
    float m = z;
    for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float ez = x == -INFINITY ? 0.0f : expf(z - m);
    const float s = wave_sum_f(ez);
    p = x == -INFINITY ? 0.0f : ez / s;
  } else if (kSig) {
    p = x == -INFINITY ? 0.0f : sigmoid(x);
  } else {
    p = x == -INFINITY ? 0.0f : expf(x - top) / sum;
  }
  return p;
}

}  // namespace moe
