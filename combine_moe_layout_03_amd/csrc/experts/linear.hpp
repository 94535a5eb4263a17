// What the dense product's kernels share: its epilogue.
#pragma once

#include "copy.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

enum Act { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSwiglu = 3 };

struct LinearEpilogue {
  const float *bias;         // nullptr: none
  const uint16_t *residual;  // nullptr: none
  void *out;                 // bf16 or float [T][N]
  uint16_t *pre;             // nullptr: not stored
  int32_t N;                 // columns of out
  bool f32;
};

// 1 / (1 + exp(-z)) and 1 / (1 + exp(z)): from the exponential that does not
// overflow, so that both keep their digits down to the smallest floats.
struct Sigmoids {
  float s, rest;
};
__device__ __forceinline__ Sigmoids sigmoids(float z) {
  const float e = expf(-fabsf(z)), big = 1.0f / (1.0f + e), small = e * big;
  return z < 0.0f ? Sigmoids{small, big} : Sigmoids{big, small};
}

template <int kAct>
__device__ __forceinline__ float activation(float z) {
  if (kAct == kActSilu || kAct == kActSwiglu) return z * sigmoids(z).s;
  // z Phi(z), from the complement so that it keeps its digits where Phi is small
  if (kAct == kActGelu) return 0.5f * z * erfcf(z * -0.70710678f);
  return z;
}

// Four columns n ... n + 3 of row t; up: the SwiGLU's second half.
template <int kAct>
__device__ __forceinline__ void linear_store(const LinearEpilogue &e, int64_t t, int n, f32x4 z,
                                             f32x4 up) {
  const int NN = kAct == kActSwiglu ? 2 * e.N : e.N;
  if (e.bias) {
    z += *reinterpret_cast<const f32x4 *>(e.bias + n);
    if (kAct == kActSwiglu) up += *reinterpret_cast<const f32x4 *>(e.bias + e.N + n);
  }
  if (kAct != kActNone && e.pre) {
    uint16_t *p = e.pre + t * NN + n;
    *reinterpret_cast<ex_u32x2 *>(p) = ex_u32x2{ex_bf16x2(z[0], z[1]), ex_bf16x2(z[2], z[3])};
    if (kAct == kActSwiglu)
      *reinterpret_cast<ex_u32x2 *>(p + e.N) =
          ex_u32x2{ex_bf16x2(up[0], up[1]), ex_bf16x2(up[2], up[3])};
  }
  f32x4 h;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    h[c] = activation<kAct>(z[c]);
    if (kAct == kActSwiglu) h[c] *= up[c];
  }
  if (e.residual) {
    const ex_u32x2 r = *reinterpret_cast<const ex_u32x2 *>(e.residual + t * e.N + n);
    h += f32x4{ex_lo(r[0]), ex_hi(r[0]), ex_lo(r[1]), ex_hi(r[1])};
  }
  if (e.f32)
    *reinterpret_cast<f32x4 *>(static_cast<float *>(e.out) + t * e.N + n) = h;
  else
    *reinterpret_cast<ex_u32x2 *>(static_cast<uint16_t *>(e.out) + t * e.N + n) =
        ex_u32x2{ex_bf16x2(h[0], h[1]), ex_bf16x2(h[2], h[3])};
}

}  // namespace moe
