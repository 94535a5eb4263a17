// The activation between an expert's two products, h = silu(gate) * up, cast
// to FP8 as moe_quantize_fp8 casts a row, and its gradient.
//
// Both are streams over the rows of the segments. How many rows those hold
// only the device knows, so every workgroup first makes the running sum of the
// E counts in LDS, then walks its share of the (row, chunk of a row) units,
// finding a unit's expert by bisection of that sum. A wave's unit is 512
// channels of h: a lane reads 8 gates and 8 ups (16 bytes each), and the 128
// channels of a scale are one 16-lane DPP row, as in the dispatch's cast. h
// stays in float up to the E4M3 code.
#include "segments.hpp"

namespace moe {
namespace {

constexpr int kSwThreads = kPlanThreads;

__device__ __forceinline__ float keep_finite(float h) {
  return fminf(fmaxf(h, -3.402823466e38f), 3.402823466e38f);
}

template <int kFlags>
__global__ __launch_bounds__(kSwThreads) void swiglu_fp8_kernel(
    Segments seg, const ex_u32x4 *__restrict__ x, ex_u32x2 *__restrict__ q,
    float *__restrict__ fscale, uint32_t *__restrict__ wscale, int32_t I, int32_t nchunk,
    int32_t *status) {
  __shared__ SegmentPlanRows plan;
  const int total = plan_segments(seg, 1, plan, status);
  const int lane = threadIdx.x & 63;
  const int nv = I / 8;  // 16-byte vectors of gates in a row
  const int64_t units = (int64_t)total * nchunk;
  const int64_t waves = (int64_t)gridDim.x * (kSwThreads / 64);
  for (int64_t u = (int64_t)blockIdx.x * (kSwThreads / 64) + (threadIdx.x >> 6); u < units;
       u += waves) {
    const int i = (int)(u / nchunk), c = (int)(u - (int64_t)i * nchunk);
    const int e = plan_find(plan, seg.E, i);
    const int64_t row = (int64_t)plan.start[e] + (i - plan.first[e]);
    const int v = c * 64 + lane;
    const bool in = v < nv;
    const ex_u32x4 *xr = x + row * 2 * nv;
    const ex_u32x4 g = xr[in ? v : 0], up = xr[nv + (in ? v : 0)];
    float h[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const float a = ex_lo(g[d]), b = ex_hi(g[d]);
      h[2 * d] = keep_finite(a / (1.0f + expf(-a)) * ex_lo(up[d]));
      h[2 * d + 1] = keep_finite(b / (1.0f + expf(-b)) * ex_hi(up[d]));
    }
    float am = 0.0f;
#pragma unroll
    for (int d = 0; d < 8; ++d) am = fmaxf(am, fabsf(h[d]));
    am = __uint_as_float(row16_max(__float_as_uint(am)));
    if (am < 1e-4f) am = 1e-4f;
    float s = am / 448.0f;
    if (kFlags & kFp8RoundScale) {
      uint32_t b = __float_as_uint(s);
      if (b & 0x7fffffu) b = (b & 0xff800000u) + 0x800000u;
      s = __uint_as_float(b);
    }
    const float y = 1.0f / s;
    float d8[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) d8[d] = fminf(fmaxf(div_by_scale(h[d], s, y), -448.0f), 448.0f);
    if (in)
      q[row * nv + v] = ex_u32x2{e4m3x4(d8[0], d8[1], d8[2], d8[3]),
                                 e4m3x4(d8[4], d8[5], d8[6], d8[7])};
    if (kFlags & kFp8Ue8m0) {
      const uint32_t word = ue8m0_word(s);
      if (lane == 0) wscale[row * nchunk + c] = word;
    } else if (in && (lane & 15) == 0) {
      fscale[row * (I / kFp8Group) + (v >> 4)] = s;
    }
  }
}

__global__ __launch_bounds__(kSwThreads) void swiglu_grad_kernel(
    Segments seg, const ex_u32x4 *x, const ex_u32x4 *__restrict__ dh, ex_u32x4 *dx, int32_t nv,
    int32_t nchunk, int32_t *status) {
  __shared__ SegmentPlanRows plan;
  const int total = plan_segments(seg, 1, plan, status);
  const int lane = threadIdx.x & 63;
  const int64_t units = (int64_t)total * nchunk;
  const int64_t waves = (int64_t)gridDim.x * (kSwThreads / 64);
  for (int64_t u = (int64_t)blockIdx.x * (kSwThreads / 64) + (threadIdx.x >> 6); u < units;
       u += waves) {
    const int i = (int)(u / nchunk), c = (int)(u - (int64_t)i * nchunk);
    const int e = plan_find(plan, seg.E, i);
    const int64_t row = (int64_t)plan.start[e] + (i - plan.first[e]);
    const int v = c * 64 + lane;
    if (v >= nv) continue;
    const int64_t at = row * 2 * nv + v;
    const ex_u32x4 g = x[at], up = x[at + nv], d = dh[row * nv + v];
    ex_u32x4 dg, du;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a[2] = {ex_lo(g[j]), ex_hi(g[j])}, b[2] = {ex_lo(up[j]), ex_hi(up[j])},
            e[2] = {ex_lo(d[j]), ex_hi(d[j])}, p[2], r[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float s = 1.0f / (1.0f + expf(-a[k]));
        p[k] = e[k] * b[k] * (s * (1.0f + a[k] * (1.0f - s)));
        r[k] = e[k] * (a[k] * s);
      }
      dg[j] = ex_bf16x2(p[0], p[1]);
      du[j] = ex_bf16x2(r[0], r[1]);
    }
    dx[at] = dg;
    dx[at + nv] = du;
  }
}

unsigned stream_blocks(const Segments &seg, int32_t nchunk) {
  const int64_t most = (seg.rows * nchunk + kSwThreads / 64 - 1) / (kSwThreads / 64);
  return (unsigned)(most < 2048 ? (most < 1 ? 1 : most) : 2048);
}

template <int kFlags>
hipError_t swiglu_k(const Segments &seg, int32_t I, const uint16_t *x, uint8_t *q, void *scale,
                    int32_t *status, hipStream_t s) {
  const int32_t nchunk = (I / 8 + 63) / 64;
  hipLaunchKernelGGL((swiglu_fp8_kernel<kFlags>), dim3(stream_blocks(seg, nchunk)),
                     dim3(kSwThreads), 0, s, seg, reinterpret_cast<const ex_u32x4 *>(x),
                     reinterpret_cast<ex_u32x2 *>(q), static_cast<float *>(scale),
                     static_cast<uint32_t *>(scale), I, nchunk, status);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu_fp8(const Segments &seg, int32_t I, const uint16_t *x, uint8_t *q,
                             void *scale, int32_t flags, int32_t *status, hipStream_t s) {
  switch (flags & (kFp8RoundScale | kFp8Ue8m0)) {  // scales are always row-major here
    case 0: return swiglu_k<0>(seg, I, x, q, scale, status, s);
    case kFp8RoundScale: return swiglu_k<kFp8RoundScale>(seg, I, x, q, scale, status, s);
    default: return swiglu_k<kFp8RoundScale | kFp8Ue8m0>(seg, I, x, q, scale, status, s);
  }
}

hipError_t launch_swiglu_grad(const Segments &seg, int32_t I, const uint16_t *x,
                              const uint16_t *dh, uint16_t *dx, int32_t *status, hipStream_t s) {
  const int32_t nv = I / 8, nchunk = (nv + 63) / 64;
  hipLaunchKernelGGL(swiglu_grad_kernel, dim3(stream_blocks(seg, nchunk)), dim3(kSwThreads), 0, s,
                     seg, reinterpret_cast<const ex_u32x4 *>(x),
                     reinterpret_cast<const ex_u32x4 *>(dh), reinterpret_cast<ex_u32x4 *>(dx), nv,
                     nchunk, status);
  return hipGetLastError();
}

}  // namespace moe
