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

// ---- tiles: segments of many rows -------------------------------------------

constexpr int kTileWaves = 8;      // 4 along the weight rows x 2 along the token rows
constexpr int kTileThreads = kTileWaves * 64;
constexpr int kTileN = 256;        // weight rows of a tile, 64 per wave
constexpr int kTileMost = 9;       // 16-row token tiles per wave
constexpr int kTileTokens = 2 * 16 * kTileMost;
constexpr int kScaleSlots = 6 * 64;  // 288 token scales (5 copies of 64), then the weights'

// Copies 16 (4) bytes per lane from global memory to LDS at base + 16 (4) * lane
// without passing registers.
__device__ __forceinline__ void copy16_to_lds(const void *src, void *base) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                   (__attribute__((address_space(3))) void *)base, 16, 0, 0);
}
__device__ __forceinline__ void copy4_to_lds(const void *src, void *base) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                   (__attribute__((address_space(3))) void *)base, 4, 0, 0);
}

__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

struct TilePos {
  int e, n0;
  int tokens;
  int64_t row0, scale_base, r_stride, g_stride;
};

// One group of 128 channels of a tile in LDS: rows of 128 bytes, the 16-byte
// chunk c of row r at chunk c ^ (r & 7), so that the 16 rows a fragment reads
// at one chunk fall on all banks.
struct TileStage {
  uint8_t w[kTileN * 128];
  uint8_t a[kTileTokens * 128];
  uint32_t scale[kScaleSlots];
};

template <int TT, bool kWords>
__device__ __forceinline__ void tile_product(const GemmArgs &ga, const TilePos &p, TileStage &st0,
                                             TileStage &st1) {
  const int lane = threadIdx.x & 63, wave = scalar(threadIdx.x >> 6);
  const int wn = wave & 3, wt = wave >> 2;
  const int C = ga.C, G = C / kFp8Group;
  const int l16 = lane & 15, quad = lane >> 4;
  const int nw = p.n0 + wn * 64;  // the wave's weight rows
  // What the wave copies of a group: 8 rows per instruction, 8 lanes a row (a
  // whole 128-byte line; 16 lanes on 16 rows, as a fragment holds them, load
  // at a quarter of the rate). Uniform bases, 32-bit lane offsets.
  constexpr int kCopies = (TT * 4 + kTileWaves - 1) / kTileWaves;
  const uint8_t *wbase = ga.w + ((int64_t)p.e * ga.N + p.n0) * C;
  const uint8_t *tbase = ga.a + p.row0 * C;
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t wo[4], to[kCopies];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (i * kTileWaves + wave) * 8 + (lane >> 3);
    wo[i] = (uint32_t)min(r, ga.N - 1 - p.n0) * (uint32_t)C + chunk;
  }
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int r = (i * kTileWaves + wave) * 8 + (lane >> 3);
    to[i] = (uint32_t)min(r, p.tokens - 1) * (uint32_t)C + chunk;
  }
  // scales of a group: waves 0-4 copy the tokens', wave 5 those of the weight rows
  const uint32_t *sbase = static_cast<const uint32_t *>(ga.a_scale) + p.scale_base;
  const int64_t so = (int64_t)min(wave * 64 + lane, p.tokens - 1) * p.r_stride;
  const float *wsbase = ga.w_scale + ((int64_t)p.e * ((ga.N + 127) / 128) + p.n0 / 128) * G;
  const int ws = (min(p.n0 + (lane & 3) * 64, ga.N - 1) / 128 - p.n0 / 128) * G;
  auto copy_group = [&](int g, TileStage &st) {
    g = min(g, G - 1);
    const int64_t k = (int64_t)g * kFp8Group;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      copy16_to_lds(wbase + k + wo[i], st.w + (i * kTileWaves + wave) * 1024);
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
      if ((i + 1) * kTileWaves <= TT * 4 || i * kTileWaves + wave < TT * 4)
        copy16_to_lds(tbase + k + to[i], st.a + (i * kTileWaves + wave) * 1024);
    if (wave < (TT + 1) / 2)
      copy4_to_lds(sbase + (kWords ? g >> 2 : g) * p.g_stride + so, st.scale + wave * 64);
    else if (wave == 5)
      copy4_to_lds(wsbase + g + ws, st.scale + 5 * 64);
  };

  f32x4 acc[4][TT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // row l16's 16 bytes at chunk quad
  const int frag0 = l16 * 128 + ((quad ^ (l16 & 7)) * 16);
  // Product q = 4 t + i (token tile t, weight rows i) is issued while product
  // q - 2 is scaled and added. The empty asm orders the two: left alone, the
  // compiler issues all products first, and their results do not fit the
  // registers.
  auto compute = [&](int g, const TileStage &st) {
    const uint8_t *wbuf = st.w + wn * 8192, *buf = st.a + wt * TT * 2048;
    const uint32_t *sc = st.scale + wt * TT * 16;
    const float b = __uint_as_float(st.scale[5 * 64 + wn]);
    auto rows16 = [&](const uint8_t *from, int t) {
      return frag(*reinterpret_cast<const ex_u32x4 *>(from + t * 2048 + frag0),
                  *reinterpret_cast<const ex_u32x4 *>(from + t * 2048 + (frag0 ^ 64)));
    };
    auto scale = [&](int t) {
      const uint32_t x = sc[t * 16 + l16];
      if (!kWords) return __uint_as_float(x);
      const uint32_t e = (x >> (8 * (g & 3))) & 255u;
      return __uint_as_float(e ? e << 23 : 0x00400000u);
    };
    i32x8 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = rows16(wbuf, i);
    f32x4 m[3];
    i32x8 a = rows16(buf, 0), next = a;
    float s = scale(0) * b, s_next = s;
#pragma unroll
    for (int q = 0; q < 4 * TT + 2; ++q) {
      const int t = q >> 2, i = q & 3;
      if (q < 4 * TT) {
        if (i == 0 && t > 0) a = next;
        if (i == 0 && t + 1 < TT) next = rows16(buf, t + 1);
        if (q >= 3) {
          f32x4 &done = acc[(q - 3) & 3][(q - 3) >> 2];
          asm volatile("" : "+v"(a), "+v"(done));
        }
        m[q % 3] = mfma_group(w[i], a);
      }
      if (q >= 2) {
        const int d = q - 2;
        f32x4 &to_add = acc[d & 3][d >> 2];
        if ((d & 3) == 0 && d > 0) s = s_next;
#pragma unroll
        for (int c = 0; c < 4; ++c) to_add[c] = __builtin_fmaf(m[d % 3][c], s, to_add[c]);
        if ((d & 3) == 0 && (d >> 2) + 1 < TT) s_next = scale((d >> 2) + 1) * b;
      }
    }
  };
  auto settle = [&]() {  // the copies of every wave have landed, the other stage is free
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    lds_barrier();
  };

  copy_group(0, st0);
  settle();
  for (int g = 0; g + 1 < G; g += 2) {  // a group past the last is copied again, not used
    copy_group(g + 1, st1);
    compute(g, st0);
    settle();
    copy_group(g + 2, st0);
    compute(g + 1, st1);
    settle();
  }
  if (G & 1) {
    compute(G - 1, st0);
    lds_barrier();
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int r = (wt * TT + t) * 16 + l16;
    if (r >= p.tokens) continue;
    uint16_t *o = ga.out + (p.row0 + r) * ga.N + nw + quad * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (nw + i * 16 + quad * 4 < ga.N)
        *reinterpret_cast<ex_u32x2 *>(o + i * 16) =
            ex_u32x2{ex_bf16x2(acc[i][t][0], acc[i][t][1]), ex_bf16x2(acc[i][t][2], acc[i][t][3])};
  }
}

template <bool kWords>
__global__ __launch_bounds__(kTileThreads, 2) void grouped_gemm_tile_kernel(Segments seg,
                                                                            GemmArgs ga) {
  __shared__ SegmentPlan plan;
  __shared__ __align__(16) TileStage st0;
  __shared__ __align__(16) TileStage st1;
  const int pieces = plan_segments<kTileThreads>(seg, kTileTokens, plan, ga.status);
  const int G = ga.C / kFp8Group, SG = kWords ? G / 4 : G;  // scale entries of a row
  const int nblk = (ga.N + kTileN - 1) / kTileN;
  // Workgroup b runs on XCD b % 8: each XCD takes one run of the tiles, so the
  // tiles in flight on it share weights and token rows in its L2.
  const int64_t tiles = (int64_t)pieces * nblk;
  const int xcd = blockIdx.x & 7, lanes = gridDim.x >> 3;
  const int64_t lo = tiles * xcd / 8, hi = tiles * (xcd + 1) / 8;
  for (int64_t u = lo + (blockIdx.x >> 3); u < hi; u += lanes) {
    TilePos p;
    // wave-uniform values, kept in scalar registers
    p.e = scalar(plan_find(plan, seg.E, (int)(u / nblk)));
    const int first = scalar(plan.first[p.e]), np = scalar(plan.first[p.e + 1]) - first;
    const int r = (int)(u - (int64_t)first * nblk);
    const int nb = scalar(r / np), piece = r - nb * np;
    const int count = scalar(seg.count[p.e]);
    const int per = scalar(((count + np - 1) / np + 31) & ~31);  // the pieces are even
    p.tokens = min(count - piece * per, per);
    p.row0 = (int64_t)scalar(plan.start[p.e]) + piece * per;
    p.n0 = nb * kTileN;
    if (seg.per_expert > 0) {
      p.scale_base = (int64_t)p.e * SG * seg.per_expert + (p.row0 - (int64_t)p.e * seg.per_expert);
      p.r_stride = 1;
      p.g_stride = seg.per_expert;
    } else {
      p.scale_base = p.row0 * SG;
      p.r_stride = SG;
      p.g_stride = 1;
    }
    switch (per >> 5) {
      case 1: case 2: tile_product<2, kWords>(ga, p, st0, st1); break;
      case 3: tile_product<3, kWords>(ga, p, st0, st1); break;
      case 4: tile_product<4, kWords>(ga, p, st0, st1); break;
      case 5: tile_product<5, kWords>(ga, p, st0, st1); break;
      case 6: tile_product<6, kWords>(ga, p, st0, st1); break;
      case 7: tile_product<7, kWords>(ga, p, st0, st1); break;
      case 8: tile_product<8, kWords>(ga, p, st0, st1); break;
      default: tile_product<9, kWords>(ga, p, st0, st1); break;
    }
  }
}

// Segments of up to this many rows are streamed, larger ones tiled.
constexpr int kStreamMost = 32;

}  // namespace

hipError_t launch_grouped_gemm(const Segments &seg, const GemmArgs &g, hipStream_t s) {
  const bool words = g.flags & kFp8Ue8m0;
  const int64_t nblk = (g.N + kRow16 - 1) / kRow16;
  const int64_t most = ((seg.rows + kStreamTokens - 1) / kStreamTokens + seg.E) * nblk;
  const unsigned grid = (unsigned)(most < 2048 ? most : 2048);
  // how many rows a segment can have at most decides which kernels are needed
  const int64_t bound = seg.max_count > 0 ? seg.max_count
                                          : (seg.per_expert > 0 ? seg.per_expert : seg.rows);
  Segments part = seg;
  part.upto = kStreamMost;
  if (words)
    hipLaunchKernelGGL((grouped_gemm_stream_kernel<true>), dim3(grid), dim3(kPlanThreads), 0, s,
                       part, g);
  else
    hipLaunchKernelGGL((grouped_gemm_stream_kernel<false>), dim3(grid), dim3(kPlanThreads), 0, s,
                       part, g);
  if (bound > kStreamMost) {
    part.over = kStreamMost;
    part.upto = 0;
    if (words)
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<true>), dim3(256), dim3(kTileThreads), 0, s,
                         part, g);
    else
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<false>), dim3(256), dim3(kTileThreads), 0, s,
                         part, g);
  }
  return hipGetLastError();
}

}  // namespace moe
