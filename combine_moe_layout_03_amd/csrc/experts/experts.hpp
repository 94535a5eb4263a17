// Internal launch interface between the C-ABI entry points (experts.hip) and
// the kernels around the experts (gate.hip, combine_grad.hip, swiglu.hip,
// grouped_gemm.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../fp8.hpp"
#include "../wave.hpp"

namespace moe {

constexpr int32_t kStBadLogit = 16;  // MOE_STATUS_BAD_LOGIT

constexpr int kGateBf16 = 1, kGateSigmoid = 2, kGateRenorm = 4;  // MOE_GATE_*

typedef uint32_t ex_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t ex_u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float ex_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float ex_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// float -> bf16 bits, round to nearest even; every NaN becomes 0x7FC0.
__device__ __forceinline__ uint32_t ex_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0x7fc0u;
  return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}
__device__ __forceinline__ uint32_t ex_bf16x2(float a, float b) {
  return ex_bf16(a) | (ex_bf16(b) << 16);
}

template <int kCtrl>
__device__ __forceinline__ float dpp_f(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)__float_as_uint(x), kCtrl, 0xf, 0xf, false));
}
__device__ __forceinline__ float lane_f(float x, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
}

// Sum over the 64 lanes, wave-uniform; the order of the additions is fixed.
__device__ __forceinline__ float wave_sum_f(float x) {
  x += dpp_f<0x128>(x);
  x += dpp_f<0x124>(x);
  x += dpp_f<0x122>(x);
  x += dpp_f<0x121>(x);
  return (lane_f(x, 0) + lane_f(x, 16)) + (lane_f(x, 32) + lane_f(x, 48));
}

// Maximum over the 64 lanes, wave-uniform: each 16-lane row's in its last lane
// (row_shr by 1, 2, 4, 8), handed on to the next row (row_bcast 15, 31).
__device__ __forceinline__ uint32_t wave_max_u(uint32_t m) {
  m = umax32(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x111, 0xf, 0xf, true));
  m = umax32(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x112, 0xf, 0xf, true));
  m = umax32(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x114, 0xf, 0xf, true));
  m = umax32(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x118, 0xf, 0xf, true));
  m = umax32(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x142, 0xa, 0xf, false));
  m = umax32(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x143, 0xc, 0xf, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)m, 63);
}

// Expert e's rows: row_start[e] ... row_start[e] + count[e] - 1, inside
// [lo, hi) where a scale layout confines them. A segment that does not fit is
// taken as empty (ok = false).
struct Segments {
  const int32_t *start, *count;
  int32_t E;
  int64_t rows;        // rows of the buffer
  int32_t per_expert;  // > 0: segment e must lie in rows [e * per_expert, (e + 1) * per_expert)
  int32_t max_count;   // > 0: no segment may hold more rows
  int32_t over, upto;  // a kernel's share: segments of more than `over`, at most `upto` rows
                       // (0: all); the one with over = 0 reports the bad segments
};

__device__ __forceinline__ int segment_rows(const Segments &s, int e, int32_t *start, bool *ok) {
  const int32_t n = s.count[e], r = s.start[e];
  *start = r;
  *ok = true;
  if (n <= 0) return 0;
  int64_t lo = 0, hi = s.rows;
  if (s.per_expert > 0) {
    lo = (int64_t)e * s.per_expert;
    hi = lo + s.per_expert;
  }
  *ok = r >= lo && (int64_t)r + n <= hi && (s.max_count <= 0 || n <= s.max_count);
  return *ok ? n : 0;
}

hipError_t launch_gate(const void *x, int32_t T, int32_t E, int32_t K, int32_t flags, float scale,
                       int64_t *idx, float *w, int32_t *status, hipStream_t s);
hipError_t launch_gate_grad(const void *x, const int64_t *idx, const float *dw, int32_t T,
                            int32_t E, int32_t K, int32_t flags, float scale, void *dx,
                            int32_t *status, hipStream_t s);

// mask.idx == nullptr: no rank mask.
hipError_t launch_combine_grad(const uint16_t *dout, const uint16_t *y, int64_t rows,
                               const int32_t *slot, const float *w, uint16_t *dy, float *dw,
                               int32_t T, int32_t K, int32_t H, const CombineMask &mask,
                               int32_t *status, hipStream_t s);

hipError_t launch_swiglu_fp8(const Segments &seg, int32_t I, const uint16_t *x, uint8_t *q,
                             void *scale, int32_t flags, int32_t *status, hipStream_t s);
hipError_t launch_swiglu_grad(const Segments &seg, int32_t I, const uint16_t *x,
                              const uint16_t *dh, uint16_t *dx, int32_t *status, hipStream_t s);

// The scale of row r, group g is at r_stride * r + g_stride * g behind the
// expert's base (row-major: the row's own scales; column-major: a column of
// the expert's rows).
struct GemmArgs {
  const uint8_t *a;
  const void *a_scale;
  const uint8_t *w;
  const float *w_scale;
  uint16_t *out;
  int32_t N, C;
  int32_t flags;
  int32_t *status;
};
hipError_t launch_grouped_gemm(const Segments &seg, const GemmArgs &g, hipStream_t s);

}  // namespace moe
