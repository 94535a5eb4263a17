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
constexpr int kWaveN = 48;         // weight rows of a wave: 3 operands of 16
constexpr int kTileN = 4 * kWaveN;  // weight rows of a tile
constexpr int kTileMost = 9;       // 16-row token tiles per wave
constexpr int kTileTokens = 2 * 16 * kTileMost;
constexpr int kScaleSlots = 6 * 64;  // 288 token scales (5 copies of 64), then the weights'

// Copies 16 (4) bytes per lane from base + off (bytes, off per lane) to LDS at
// byte `to` + 16 (4) * lane without passing registers. Written in asm because
// the compiler, not knowing which buffer a copy in flight writes, would wait
// for all copies before any LDS read; the loop below counts them itself. No
// register is written, so nothing can be reused too early.
__device__ __forceinline__ void copy16_to_lds(const void *base, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(to), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void copy4_to_lds(const void *base, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :: "s"(to), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_byte(const void *p) {  // address of a shared object
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// Wave-uniform values, moved to scalar registers.
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }
template <class T>
__device__ __forceinline__ T *scalar(T *x) {
  const uint64_t v = (uint64_t)(uintptr_t)x;
  return (T *)(uintptr_t)((uint64_t)(uint32_t)scalar((int)(uint32_t)v) |
                          (uint64_t)(uint32_t)scalar((int)(uint32_t)(v >> 32)) << 32);
}

struct TilePos {
  int e, n0;
  int tokens;
  int64_t row0, scale_base, r_stride, g_stride;
};

// Groups of 128 channels of a tile in LDS: rows of 128 bytes, the 16-byte
// chunk c of row r at chunk c ^ (r & 7), so that the 16 rows a fragment reads
// at one chunk fall on all banks. The weights come from HBM and are copied two
// groups ahead into three buffers, the token rows (in L2 after the first tile
// of an expert) one group ahead into two.
struct TileRows {
  uint8_t a[kTileTokens * 128];
  uint32_t scale[kScaleSlots];
};
struct TileBuffers {
  uint8_t w[3][kTileN * 128];
  TileRows rows[2];
};

template <int TT, bool kWords>
__device__ __forceinline__ void tile_product(const GemmArgs &ga, const TilePos &p,
                                             TileBuffers &lds) {
  const int lane = threadIdx.x & 63, wave = scalar(threadIdx.x >> 6);
  const int wn = wave & 3, wt = wave >> 2;
  const int C = ga.C, G = C / kFp8Group;
  const int l16 = lane & 15, quad = lane >> 4;
  const int nw = p.n0 + wn * kWaveN;  // the wave's weight rows
  // What the wave copies of a group: 8 rows per instruction, 8 lanes a row (a
  // whole 128-byte line; 16 lanes on 16 rows, as a fragment holds them, load
  // at a quarter of the rate). Uniform bases, 32-bit lane offsets.
  constexpr int kCopies = (TT * 4 + kTileWaves - 1) / kTileWaves;
  const uint8_t *wbase = scalar(ga.w + ((int64_t)p.e * ga.N + p.n0) * C);
  const uint8_t *tbase = scalar(ga.a + p.row0 * C);
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t wo[3], to_off[kCopies];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int r = (i * kTileWaves + wave) * 8 + (lane >> 3);
    wo[i] = (uint32_t)min(r, ga.N - 1 - p.n0) * (uint32_t)C + chunk;
  }
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int r = (i * kTileWaves + wave) * 8 + (lane >> 3);
    to_off[i] = (uint32_t)min(r, p.tokens - 1) * (uint32_t)C + chunk;
  }
  // scales of a group: waves 0-4 copy the tokens', wave 5 those of the weight
  // rows, one for each 16
  const uint32_t *sbase = scalar(static_cast<const uint32_t *>(ga.a_scale) + p.scale_base);
  const uint32_t so = (uint32_t)min(wave * 64 + lane, p.tokens - 1) * (uint32_t)p.r_stride * 4;
  const float *wsbase =
      scalar(ga.w_scale + ((int64_t)p.e * ((ga.N + 127) / 128) + p.n0 / 128) * G);
  const uint32_t ws =
      (uint32_t)(min(p.n0 + min(lane, 11) * 16, ga.N - 1) / 128 - p.n0 / 128) * (uint32_t)G * 4;
  const uint32_t lds_w = lds_byte(lds.w) + wave * 1024, lds_a = lds_byte(lds.rows) + wave * 1024;
  const uint32_t lds_s = lds_byte(lds.rows[0].scale) + min(wave, 5) * 256;
  auto copy_weights = [&](int g, int to) {
    const uint8_t *b = wbase + (int64_t)min(g, G - 1) * kFp8Group;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      copy16_to_lds(b, wo[i], lds_w + to * (kTileN * 128) + i * kTileWaves * 1024);
  };
  auto copy_rows = [&](int g, int to) {
    g = min(g, G - 1);
    const uint8_t *b = tbase + (int64_t)g * kFp8Group;
    const uint32_t at = lds_a + to * (uint32_t)sizeof(TileRows);
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
      if ((i + 1) * kTileWaves <= TT * 4 || i * kTileWaves + wave < TT * 4)
        copy16_to_lds(b, to_off[i], at + i * kTileWaves * 1024);
    const uint32_t st = lds_s + to * (uint32_t)sizeof(TileRows);
    if (wave < (TT + 1) / 2)
      copy4_to_lds(sbase + (kWords ? g >> 2 : g) * p.g_stride, so, st);
    else if (wave == 5)
      copy4_to_lds(wsbase + g, ws, st);
  };

  f32x4 acc[3][TT];
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // row l16's 16 bytes at chunk quad
  const int frag0 = l16 * 128 + ((quad ^ (l16 & 7)) * 16);
  // Product q = 3 t + i (token tile t, weight rows i) is issued while product
  // q - 2 is scaled and added. The empty asm orders the two: left alone, the
  // compiler issues all products first, and their results do not fit the
  // registers.
  auto compute = [&](int g, const uint8_t *sw, const TileRows &sa) {
    const uint8_t *wbuf = sw + wn * kWaveN * 128, *buf = sa.a + wt * TT * 2048;
    const uint32_t *sc = sa.scale + wt * TT * 16;
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
    i32x8 w[3];
    float b[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      w[i] = rows16(wbuf, i);
      b[i] = __uint_as_float(sa.scale[5 * 64 + wn * 3 + i]);
    }
    f32x4 m[3];
    i32x8 a = rows16(buf, 0), next = a;
    float s = scale(0), s_next = s;
#pragma unroll
    for (int q = 0; q < 3 * TT + 2; ++q) {
      const int t = q / 3, i = q % 3;
      if (q < 3 * TT) {
        if (i == 0 && t > 0) a = next;
        if (i == 0 && t + 1 < TT) next = rows16(buf, t + 1);
        if (q >= 3) {
          f32x4 &done = acc[i][t - 1];
          asm volatile("" : "+v"(a), "+v"(done));
        }
        m[i] = mfma_group(w[i], a);
      }
      if (q >= 2) {
        const int d = q - 2, dt = d / 3, di = d % 3;
        if (di == 0 && d > 0) s = s_next;
        const float f = s * b[di];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[di][dt][c] = __builtin_fmaf(m[di][c], f, acc[di][dt][c]);
        if (di == 0 && dt + 1 < TT) s_next = scale(dt + 1);
      }
    }
  };
  // While a group is computed, the next group's token rows and the weights of
  // the group after that are on their way. At its end all copies but those
  // last three of each wave have landed, for every wave. Groups past the last
  // are copied again, not used.
  copy_rows(0, 0);
  copy_weights(0, 0);
  copy_weights(1, 1);
  __builtin_amdgcn_s_waitcnt(0x0f73);  // vmcnt(3)
  lds_barrier();
  int w_now = 0, w_free = 2;
  for (int g = 0; g < G; ++g) {
    copy_rows(g + 1, (g + 1) & 1);
    copy_weights(g + 2, w_free);
    compute(g, lds.w[w_now], lds.rows[g & 1]);
    w_free = w_now;
    w_now = w_now == 2 ? 0 : w_now + 1;
    __builtin_amdgcn_s_waitcnt(0x0f73);
    lds_barrier();
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // the last copies land before the buffers are used again
  lds_barrier();
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int r = (wt * TT + t) * 16 + l16;
    if (r >= p.tokens) continue;
    uint16_t *o = ga.out + (p.row0 + r) * ga.N + nw + quad * 4;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (nw + i * 16 + quad * 4 < ga.N)
        *reinterpret_cast<ex_u32x2 *>(o + i * 16) =
            ex_u32x2{ex_bf16x2(acc[i][t][0], acc[i][t][1]), ex_bf16x2(acc[i][t][2], acc[i][t][3])};
  }
}

template <bool kWords>
__global__ __launch_bounds__(kTileThreads, 2) void grouped_gemm_tile_kernel(Segments seg,
                                                                            GemmArgs ga) {
  __shared__ SegmentPlan plan;
  __shared__ __align__(16) TileBuffers lds;
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
    const int r = scalar((int)(u - (int64_t)first * nblk));
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
      case 1: case 2: tile_product<2, kWords>(ga, p, lds); break;
      case 3: tile_product<3, kWords>(ga, p, lds); break;
      case 4: tile_product<4, kWords>(ga, p, lds); break;
      case 5: tile_product<5, kWords>(ga, p, lds); break;
      case 6: tile_product<6, kWords>(ga, p, lds); break;
      case 7: tile_product<7, kWords>(ga, p, lds); break;
      case 8: tile_product<8, kWords>(ga, p, lds); break;
      default: tile_product<9, kWords>(ga, p, lds); break;
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
