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
//
// Bound by bytes: 65536 rows of 2 x 2048, the cast 675 MB in 132 us and the gradient
// 1342 MB in 258, the two calls 383 us (5.3 TB/s; a large copy reaches 6.1). The
// cast was bound by instructions (268 per unit of 512 channels) until the walk's
// addresses were left to the scalar unit and the sigmoid was cut to what its error
// allows (181 now; the codes' exact quotients cost 3 us against h times the scale's
// reciprocal). Rows in runs, because a wave then looks a segment
// up only when it leaves one: units strided over the whole grid take 394 us;
// twice the grid, or two units' registers in turn, change nothing, half the grid
// costs 2%, loads or stores not marked nontemporal 3%. 512 rows in 256 stripes:
// 4.8 us, most of it the launch and the sum of the counts (8.0 with the run split
// by 64-bit divisions, which take 2 us of a workgroup's start each).
#include "cast.hpp"
#include "segments.hpp"

namespace moe {
namespace {

constexpr int kSwThreads = kPlanThreads;
// Whether one of a vector's eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool any_not_finite(ex_u32x4 v) {
  bool r = false;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r = r || (v[j] & 0x7f80u) == 0x7f80u || (v[j] & 0x7f800000u) == 0x7f800000u;
  return r;
}

// 4 / (1 + exp(-x)) of a bf16 value within six half float steps for |x| <= 88.5
// (one step each for the exponential and the reciprocal, half for the sum and the
// correction); beyond, 0 or 4. 2^t with t = -x log2(e) rounded to one float would
// be off by 2^-24 |x|: what t ln2 differs from -x (ln2 in two floats; exact to
// 2^-40) is added back. At the bound -89 the power is infinite and the correction
// positive, so the result is 0; a bf16 value inside has a finite power. Four times
// the sigmoid, because the reciprocal flushes subnormals, which the sigmoid of
// -87.5 to -88.5 is and its product with x is not; callers take x / 4 or such.
__device__ __forceinline__ float sigmoid4_of(float x) {
  constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Low = -1.90465430e-9f;
  x = __builtin_amdgcn_fmed3f(x, -89.0f, 89.0f);
  const float t = x * -kLog2e;
  const float d = __builtin_fmaf(-t, kLn2Low, __builtin_fmaf(-t, kLn2, -x));
  const float e0 = __builtin_amdgcn_exp2f(t);
  return __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fmaf(e0, d, e0), 0.25f, 0.25f));
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The rows of all segments, cut evenly into one run per workgroup; its waves
// take the run's (row, 512-channel chunk) units in turn. A run's rows ascend,
// so a wave finds the first one's expert by bisection and steps on from there.
struct RowWalk {
  int e, lo, hi;  // expert, its rows [lo, hi) among all rows
  int64_t start;
  __device__ __forceinline__ void at(const SegmentPlanRows &p, int i) {
    if (i < hi) return;
    while (i >= uniform(p.first[e + 1])) ++e;
    set(p);
  }
  __device__ __forceinline__ void find(const SegmentPlanRows &p, int E, int i) {
    e = plan_find(p, E, i);
    set(p);
  }
  __device__ __forceinline__ void set(const SegmentPlanRows &p) {
    e = uniform(e);
    lo = uniform(p.first[e]);
    hi = uniform(p.first[e + 1]);
    start = uniform(p.start[e]);
  }
  __device__ __forceinline__ int64_t row(int i) const { return start + (i - lo); }
};

// Runs body(row, chunk of the row) for the wave's units; load(row, chunk) is
// called one unit ahead and its result handed to body.
template <class Load, class Body>
__device__ __forceinline__ void for_rows(const Segments &seg, const SegmentPlanRows &plan,
                                         int total, int nchunk, Load load, Body body) {
  // All of the walk is the same in every lane. Divisions are done in vector
  // registers: read back, they leave it and every address it makes to the scalar
  // unit.
  const int wave = uniform(threadIdx.x >> 6);
  constexpr int kWaves = kSwThreads / 64;
  const int each = uniform((uint32_t)total / gridDim.x), rest = total - each * (int)gridDim.x;
  const int r0 = uniform(each * (int)blockIdx.x + min((int)blockIdx.x, rest));
  const int r1 = uniform(r0 + each + ((int)blockIdx.x < rest ? 1 : 0));
  const int skip = uniform(wave / nchunk);
  int i = r0 + skip, c = wave - skip * nchunk;  // unit: row i, chunk c
  if (i >= r1) return;
  RowWalk walk;
  walk.find(plan, seg.E, i);
  int64_t row = walk.row(i);
  auto v = load(row, c);
  while (true) {
    int ni = i, nc = c + kWaves;
    while (nc >= nchunk) {
      nc -= nchunk;
      ++ni;
    }
    const bool more = ni < r1;
    int64_t next = row;
    auto nv = v;
    if (more) {
      walk.at(plan, ni);
      next = walk.row(ni);
      nv = load(next, nc);
    }
    body(row, c, v);
    if (!more) return;
    v = nv;
    row = next;
    i = ni;
    c = nc;
  }
}

struct GateUp {
  ex_u32x4 g, u;
};

template <int kFlags>
__global__ __launch_bounds__(kSwThreads) void swiglu_fp8_kernel(
    Segments seg, const ex_u32x4 *__restrict__ x, ex_u32x2 *__restrict__ q,
    float *__restrict__ fscale, uint32_t *__restrict__ wscale, int32_t I, int32_t nchunk,
    int32_t *status) {
  __shared__ SegmentPlanRows plan;
  const int total = uniform(plan_segments(seg, 1, plan, status));
  const int lane = threadIdx.x & 63;
  const int nv = I / 8;  // 16-byte vectors of gates in a row
  auto load = [&](int64_t row, int c) {
    const uint32_t v = (uint32_t)min(c * 64 + lane, nv - 1);
    const ex_u32x4 *xr = x + row * 2 * nv;
    return GateUp{__builtin_nontemporal_load(xr + v), __builtin_nontemporal_load(xr + nv + v)};
  };
  for_rows(seg, plan, total, nchunk, load, [&](int64_t row, int c, const GateUp &in) {
    const int v = c * 64 + lane;
    const bool ok = v < nv;
    float h[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const float a = ex_lo(in.g[d]), b = ex_hi(in.g[d]);
      h[2 * d] = 0.25f * a * sigmoid4_of(a) * ex_lo(in.u[d]);
      h[2 * d + 1] = 0.25f * b * sigmoid4_of(b) * ex_hi(in.u[d]);
    }
    // The lane's largest |h| (NaN if one is, unlike fmaxf), over the group as bit
    // patterns, whose integer order puts infinities and NaN on top. A gate or up
    // that is not finite leaves an h that is not.
    uint32_t top = row16_max(largest(h));
    bool spoilt = false;
    if (__ballot(top >= kInfBits)) {  // uniform, and rare
      // A product of finite values past the float range is kept at the largest
      // float; a group with an input that is not finite gets the scale NaN and, by
      // the quotients with it, NaN codes.
      const bool mine = any_not_finite(in.g) || any_not_finite(in.u);
#pragma unroll
      for (int d = 0; d < 8; ++d) h[d] = keep_finite(h[d]);
      top = row16_max(mine ? kInfBits : largest(h));
      spoilt = top >= kInfBits;
    }
    const float sc = group_scale<kFlags>(top, spoilt);
    const ex_u32x2 codes = group_codes(h, sc);
    if (ok)
      __builtin_nontemporal_store(codes, q + row * nv + v);
    if (kFlags & kFp8Ue8m0) {
      const uint32_t word = ue8m0_word(sc);
      if (lane == 0) wscale[row * nchunk + c] = word;
    } else if (ok && (lane & 15) == 0) {
      fscale[row * (I / kFp8Group) + (v >> 4)] = sc;
    }
  });
}

struct GateUpGrad {
  ex_u32x4 g, u, d;
};

__global__ __launch_bounds__(kSwThreads) void swiglu_grad_kernel(
    Segments seg, const ex_u32x4 *x, const ex_u32x4 *__restrict__ dh, ex_u32x4 *dx, int32_t nv,
    int32_t nchunk, int32_t *status) {
  __shared__ SegmentPlanRows plan;
  const int total = uniform(plan_segments(seg, 1, plan, status));
  const int lane = threadIdx.x & 63;
  // (x may be dx: a unit's vectors are read before they are written, and by no
  // other wave)
  auto load = [&](int64_t row, int c) {
    const uint32_t v = (uint32_t)min(c * 64 + lane, nv - 1);
    const ex_u32x4 *xr = x + row * 2 * nv;
    return GateUpGrad{__builtin_nontemporal_load(xr + v), __builtin_nontemporal_load(xr + nv + v),
                      __builtin_nontemporal_load(dh + row * nv + v)};
  };
  for_rows(seg, plan, total, nchunk, load, [&](int64_t row, int c, const GateUpGrad &in) {
    const int v = c * 64 + lane;
    if (v >= nv) return;
    ex_u32x4 dg, du;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a[2] = {ex_lo(in.g[j]), ex_hi(in.g[j])}, b[2] = {ex_lo(in.u[j]), ex_hi(in.u[j])},
            e[2] = {ex_lo(in.d[j]), ex_hi(in.d[j])}, p[2], r[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float s4 = sigmoid4_of(a[k]), a4 = 0.25f * a[k];
        const float slope = s4 * __builtin_fmaf(a4, __builtin_fmaf(s4, -0.25f, 1.0f), 0.25f);
        // The larger factor first: d_h * u can pass the float range, and u times a
        // small slope fall below it, where the product of the three does not. The
        // slope is at most 1.1, so half of it keeps the first product in range
        // too; a power of two, it changes no rounding.
        const bool up = fabsf(b[k]) > fabsf(e[k]);
        const float big = up ? b[k] : e[k], small = up ? e[k] : b[k];
        p[k] = 2.0f * (small * (big * (0.5f * slope)));
        r[k] = e[k] * (a4 * s4);
      }
      dg[j] = ex_bf16x2(p[0], p[1]);
      du[j] = ex_bf16x2(r[0], r[1]);
    }
    const int64_t at = row * 2 * nv + v;
    __builtin_nontemporal_store(dg, dx + at);
    __builtin_nontemporal_store(du, dx + at + nv);
  });
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
