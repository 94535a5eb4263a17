// The experts' products on FP8 rows:
//   out[r][n] = sum_g a_scale(r, g) * w_scale[e][n / 128][g] * <a[r], w[e][n]> over group g,
// groups of 128 channels, for the rows r of expert e's segment.
//
// One matrix instruction (16 x 16 x 128, E4M3 operands, float result) covers a
// whole group of 16 weight rows and 16 token rows, so each result is scaled
// once and added to a float accumulator: t = W * A^T, acc += t * (sa * sb).
// With the weights as first operand a lane's four results share one token, so
// its scale is one number per lane, and the weights' scale is one per wave.
// Both operands are read in the same channel order within the group, which is
// all the sum needs: lane l holds channels 16 (l / 16) ... + 15 and the same 64
// further of row l % 16.
#include "segments.hpp"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRow16 = 16;          // rows of a matrix instruction's operand
constexpr int kStreamTokens = 64;   // token rows of a unit
constexpr int kStreamWaves = 4;

__device__ __forceinline__ i32x8 frag(ex_u32x4 lo, ex_u32x4 hi) {
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}
__device__ __forceinline__ f32x4 mfma_group(i32x8 w, i32x8 a) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, 0, 0, 0);
}

// A float scale, or exponent byte g % 4 of a packed word.
template <bool kWords>
__device__ __forceinline__ float row_scale(const void *p, int64_t base, int64_t g_stride, int g) {
  if (kWords) {
    const uint32_t w = static_cast<const uint32_t *>(p)[base + (g >> 2) * g_stride];
    const uint32_t b = (w >> (8 * (g & 3))) & 255u;
    return __uint_as_float(b ? b << 23 : 0x00400000u);
  }
  return static_cast<const float *>(p)[base + g * g_stride];
}

struct StreamShared {
  SegmentPlan plan;
  float part[kStreamWaves][kStreamTokens][kRow16 + 1];
};

// One unit: 16 weight rows n0 ... n0 + 15, TT * 16 token rows. The waves share
// the channels out, group by group, and join their sums in LDS.
template <int TT, bool kWords>
__device__ __forceinline__ void stream_unit(const GemmArgs &ga, StreamShared &sh, int e, int n0,
                                            int64_t row0, int tokens, int64_t scale_base,
                                            int64_t r_stride, int64_t g_stride) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int C = ga.C, G = C / kFp8Group;
  const int l16 = lane & 15, c16 = (lane >> 4) * 16;
  const int n = min(n0 + l16, ga.N - 1);
  const uint8_t *wp = ga.w + ((int64_t)e * ga.N + n) * C + c16;
  const float *sb = ga.w_scale + ((int64_t)e * ((ga.N + 127) / 128) + n0 / 128) * G;
  const uint8_t *ap[TT];
  int64_t as[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t r = min(t * 16 + l16, tokens - 1);
    ap[t] = ga.a + (row0 + r) * C + c16;
    as[t] = scale_base + r * r_stride;
  }
  f32x4 acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = TT == 1 ? 4 : 2;  // groups in flight
  for (int g0 = wave; g0 < G; g0 += U * kStreamWaves) {
    ex_u32x4 w0[U], w1[U], a0[U][TT], a1[U][TT];
    float s[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = min(g0 + u * kStreamWaves, G - 1);
      const int64_t k = (int64_t)g * kFp8Group;
      w0[u] = *reinterpret_cast<const ex_u32x4 *>(wp + k);
      w1[u] = *reinterpret_cast<const ex_u32x4 *>(wp + k + 64);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        a0[u][t] = *reinterpret_cast<const ex_u32x4 *>(ap[t] + k);
        a1[u][t] = *reinterpret_cast<const ex_u32x4 *>(ap[t] + k + 64);
        s[u][t] = row_scale<kWords>(ga.a_scale, as[t], g_stride, g);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * kStreamWaves;
      if (g >= G) break;
      const float b = sb[g];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const f32x4 p = mfma_group(frag(w0[u], w1[u]), frag(a0[u][t], a1[u][t]));
        const float sc = s[u][t] * b;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(p[i], sc, acc[t][i]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) sh.part[wave][t * 16 + l16][(lane >> 4) * 4 + i] = acc[t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * 8; i += kPlanThreads) {
    const int t = i >> 3, c = (i & 7) * 2;
    float v[2];
#pragma unroll
    for (int d = 0; d < 2; ++d)
      v[d] = (sh.part[0][t][c + d] + sh.part[1][t][c + d]) +
             (sh.part[2][t][c + d] + sh.part[3][t][c + d]);
    if (n0 + c < ga.N)
      *reinterpret_cast<uint32_t *>(ga.out + (row0 + t) * ga.N + n0 + c) = ex_bf16x2(v[0], v[1]);
  }
  __syncthreads();
}

template <bool kWords>
__global__ __launch_bounds__(kPlanThreads) void grouped_gemm_stream_kernel(Segments seg,
                                                                           GemmArgs ga) {
  __shared__ StreamShared sh;
  const int pieces = plan_segments(seg, kStreamTokens, sh.plan, ga.status);
  const int G = ga.C / kFp8Group, SG = kWords ? G / 4 : G;  // scale entries of a row
  const int nblk = (ga.N + kRow16 - 1) / kRow16;
  const int64_t units = (int64_t)pieces * nblk;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = (int)(u / nblk), nb = (int)(u - (int64_t)i * nblk);
    const int e = plan_find(sh.plan, seg.E, i);
    const int t0 = (i - sh.plan.first[e]) * kStreamTokens;
    const int tokens = min(seg.count[e] - t0, kStreamTokens);
    const int64_t row0 = (int64_t)sh.plan.start[e] + t0;
    int64_t base, rs, gs;
    if (seg.per_expert > 0) {
      base = (int64_t)e * SG * seg.per_expert + (row0 - (int64_t)e * seg.per_expert);
      rs = 1;
      gs = seg.per_expert;
    } else {
      base = row0 * SG;
      rs = SG;
      gs = 1;
    }
    if (tokens <= 16)
      stream_unit<1, kWords>(ga, sh, e, nb * kRow16, row0, tokens, base, rs, gs);
    else if (tokens <= 32)
      stream_unit<2, kWords>(ga, sh, e, nb * kRow16, row0, tokens, base, rs, gs);
    else
      stream_unit<4, kWords>(ga, sh, e, nb * kRow16, row0, tokens, base, rs, gs);
  }
}

}  // namespace

hipError_t launch_grouped_gemm(const Segments &seg, const GemmArgs &g, hipStream_t s) {
  const int64_t nblk = (g.N + kRow16 - 1) / kRow16;
  const int64_t most = ((seg.rows + kStreamTokens - 1) / kStreamTokens + seg.E) * nblk;
  const unsigned grid = (unsigned)(most < 2048 ? most : 2048);
  if (g.flags & kFp8Ue8m0)
    hipLaunchKernelGGL((grouped_gemm_stream_kernel<true>), dim3(grid), dim3(kPlanThreads), 0, s,
                       seg, g);
  else
    hipLaunchKernelGGL((grouped_gemm_stream_kernel<false>), dim3(grid), dim3(kPlanThreads), 0, s,
                       seg, g);
  return hipGetLastError();
}

}  // namespace moe
