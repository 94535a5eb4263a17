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

// 1 / (1 + exp(-z)) and 1 / (1 + exp(z)), from the exponential that does not
// overflow, the square of its root, so that both keep their digits down to the
// smallest floats: off by |z| half float steps (the exponent's rounding) and 8 (two
// steps of the root, the reciprocal, and two products).
struct Sigmoids {
  float s, rest;
};
__device__ __forceinline__ Sigmoids sigmoids(float z) {
  const float root = __builtin_amdgcn_exp2f(fabsf(z) * -0.72134752f), e = root * root;
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  return z < 0.0f ? Sigmoids{small, big} : Sigmoids{big, small};
}

// The normal law: its distribution function and its density at z. With x = |z| the
// tail is exp(-x^2 / 2) times a function of x that falls slowly, a polynomial of
// degree 8 in 1 / (1 + 0.23 x), fitted by least relative error over 0 <= x <= 13.5:
// 4.8e-8 off. With its rounding 16 half float steps, and z^2 more of the exponent's.
struct Normal {
  float below, density;
};
__device__ __forceinline__ Normal normal(float z) {
  const float e = __builtin_amdgcn_exp2f(z * z * -0.72134752f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(z), 0.23f, 1.0f));
  float q = -0.0784352568f;
  q = __builtin_fmaf(q, t, 0.290248429f);
  q = __builtin_fmaf(q, t, -0.277762615f);
  q = __builtin_fmaf(q, t, 0.301026458f);
  q = __builtin_fmaf(q, t, -0.0325876084f);
  q = __builtin_fmaf(q, t, 0.119359958f);
  q = __builtin_fmaf(q, t, 0.0858062026f);
  q = __builtin_fmaf(q, t, 0.0923717272f);
  q = __builtin_fmaf(q, t, -2.73195771e-05f);
  const float tail = e * q;
  return {z < 0.0f ? tail : 1.0f - tail, 0.39894228f * e};
}

template <int kAct>
__device__ __forceinline__ float activation(float z) {
  if (kAct == kActSilu || kAct == kActSwiglu) return z * sigmoids(z).s;
  if (kAct == kActGelu) return z * normal(z).below;
  return z;
}

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 two_of(const float *p) {  // 16-byte aligned
  const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ ex_u32x4 bf16_of(f32x8 v) {
  return ex_u32x4{ex_round2(v[0], v[1]), ex_round2(v[2], v[3]), ex_round2(v[4], v[5]),
                  ex_round2(v[6], v[7])};
}

// The residual of eight columns n ... n + 7 of row t, to be loaded ahead.
__device__ __forceinline__ ex_u32x4 linear_residual(const LinearEpilogue &e, int64_t t, int n) {
  return e.residual ? *reinterpret_cast<const ex_u32x4 *>(e.residual + t * e.N + n)
                    : ex_u32x4{0, 0, 0, 0};
}

// Those columns from their sums; up: the SwiGLU's second half.
template <int kAct>
__device__ __forceinline__ void linear_store(const LinearEpilogue &e, int64_t t, int n, f32x8 z,
                                             f32x8 up, ex_u32x4 residual) {
  const int NN = kAct == kActSwiglu ? 2 * e.N : e.N;
  if (e.bias) {
    z += two_of(e.bias + n);
    if (kAct == kActSwiglu) up += two_of(e.bias + e.N + n);
  }
  if (kAct != kActNone && e.pre) {
    uint16_t *p = e.pre + t * NN + n;
    *reinterpret_cast<ex_u32x4 *>(p) = bf16_of(z);
    if (kAct == kActSwiglu) *reinterpret_cast<ex_u32x4 *>(p + e.N) = bf16_of(up);
  }
  f32x8 h;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    h[c] = activation<kAct>(z[c]);
    if (kAct == kActSwiglu) h[c] *= up[c];
  }
  if (e.residual) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      h[2 * c] += ex_lo(residual[c]);
      h[2 * c + 1] += ex_hi(residual[c]);
    }
  }
  if (e.f32) {
    float *o = static_cast<float *>(e.out) + t * e.N + n;
    *reinterpret_cast<f32x4 *>(o) = f32x4{h[0], h[1], h[2], h[3]};
    *reinterpret_cast<f32x4 *>(o + 4) = f32x4{h[4], h[5], h[6], h[7]};
  } else {
    *reinterpret_cast<ex_u32x4 *>(static_cast<uint16_t *>(e.out) + t * e.N + n) = bf16_of(h);
  }
}

// The same for four columns.
template <int kAct>
__device__ __forceinline__ void linear_store4(const LinearEpilogue &e, int64_t t, int n, f32x4 z,
                                              f32x4 up) {
  const int NN = kAct == kActSwiglu ? 2 * e.N : e.N;
  if (e.bias) {
    z += *reinterpret_cast<const f32x4 *>(e.bias + n);
    if (kAct == kActSwiglu) up += *reinterpret_cast<const f32x4 *>(e.bias + e.N + n);
  }
  if (kAct != kActNone && e.pre) {
    uint16_t *p = e.pre + t * NN + n;
    *reinterpret_cast<ex_u32x2 *>(p) = ex_u32x2{ex_round2(z[0], z[1]), ex_round2(z[2], z[3])};
    if (kAct == kActSwiglu)
      *reinterpret_cast<ex_u32x2 *>(p + e.N) =
          ex_u32x2{ex_round2(up[0], up[1]), ex_round2(up[2], up[3])};
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
        ex_u32x2{ex_round2(h[0], h[1]), ex_round2(h[2], h[3])};
}

}  // namespace moe
