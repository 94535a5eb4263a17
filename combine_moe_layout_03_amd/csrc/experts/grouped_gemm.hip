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

__device__ __forceinline__ i32x8 frag(ex_u32x4 lo, ex_u32x4 hi) {
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}
__device__ __forceinline__ f32x4 mfma_group(i32x8 w, i32x8 a) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, 0, 0, 0);
}

// Wave-uniform values, moved to scalar registers.
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }
template <class T>
__device__ __forceinline__ T *scalar(T *x) {
  const uint64_t v = (uint64_t)(uintptr_t)x;
  return (T *)(uintptr_t)((uint64_t)(uint32_t)scalar((int)(uint32_t)v) |
                          (uint64_t)(uint32_t)scalar((int)(uint32_t)(v >> 32)) << 32);
}

// Copies 16 (4) bytes per lane from base + off (bytes, off per lane) to LDS at
// byte `to` + 16 (4) * lane without passing registers. Written in asm because
// the compiler, not knowing which buffer a copy in flight writes, would wait
// for all copies before any LDS read; the loop below counts them itself. No
// register is written, so nothing can be reused too early.
__device__ __forceinline__ void copy16_to_lds(const void *base, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(scalar((int)to)), "v"(off), "s"(scalar(base)) : "memory", "m0");
}
// The same for bytes that nobody reads again: marked to leave L2 first.
__device__ __forceinline__ void copy16_once(const void *base, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
               :: "s"(scalar((int)to)), "v"(off), "s"(scalar(base)) : "memory", "m0");
}
__device__ __forceinline__ void copy4_to_lds(const void *base, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :: "s"(scalar((int)to)), "v"(off), "s"(scalar(base)) : "memory", "m0");
}
// The same with an address per lane.
__device__ __forceinline__ void copy4_to_lds_at(const void *from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :: "s"(scalar((int)to)), "v"(from) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_byte(const void *p) {  // address of a shared object
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// Rows of 128 bytes (a group) in LDS, the 16-byte chunk c of row r at chunk
// c ^ (r & 7), so that the 16 rows a fragment reads at one chunk fall on all
// banks. A copy moves 8 rows, 8 lanes a row: whole lines. (16 lanes on 16 rows,
// as a fragment holds them, load at 16 bytes a clock and CU from L2 instead of
// 55.) The lane's bytes of rows t * 16 ... t * 16 + 15:
__device__ __forceinline__ i32x8 rows16(const uint8_t *rows, int t) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
  const int at = t * 2048 + l16 * 128 + ((quad ^ (l16 & 7)) * 16);
  return frag(*reinterpret_cast<const ex_u32x4 *>(rows + at),
              *reinterpret_cast<const ex_u32x4 *>(rows + (at ^ 64)));
}
// The value of exponent byte e of a UE8M0 word.
__device__ __forceinline__ float byte_scale(uint32_t word, int e) {
  const uint32_t b = (word >> (8 * e)) & 255u;
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// ---- stream: segments of few rows -------------------------------------------
//
// Few rows per expert make this a read of the weights. A unit is 32 weight rows
// x up to 16 token rows, and every wave streams units of its own through a ring
// of three groups in its own part of LDS, without a barrier: the copies of the
// third group, also of the next unit, are in flight while the first is
// multiplied. With fewer units than half the waves on the chip the eight waves
// of a workgroup share a unit's groups out instead and join their sums in LDS.
//
// Bound by the weights' bytes, which every unit reads once. 16 tokens x 8 of 256
// experts, 7168 channels to 4096: 451 us for 2996 MB (6.6 TB/s; a copy, half
// reads and half writes, reaches 6.1); 128 tokens x 8, 2048 to 7168: 583 us
// for 3711 MB (6.4 TB/s). The weights' copies marked to leave L2 first took these
// from 506 and 670 us. A token alone (8 experts, 7168 to 4096): 43 us, 5.5 TB/s.

constexpr int kStreamTokens = 16;  // most token rows of a unit
constexpr int kStreamN = 32;       // weight rows of a unit
constexpr int kStreamWaves = 8;
constexpr int kStreamThreads = kStreamWaves * 64;
constexpr int kStreamRing = 3;
constexpr int kStreamCopies = kStreamN / 8 + kStreamTokens / 8 + 1;  // of a group

struct StreamStage {
  uint8_t w[kStreamN * 128];
  uint8_t a[kStreamTokens * 128];
  uint32_t scale[64];  // lanes 0-15: the tokens', lane 16: the weights'
};
struct StreamShared {
  StreamStage ring[kStreamWaves][kStreamRing];
  SegmentPlanRows plan;
};
static_assert(sizeof(float) * kStreamN * (kStreamTokens + 1) <= sizeof(StreamStage) * kStreamRing,
              "a wave's partial sums take the place of its ring");

struct StreamUnit {
  int e, n0, tokens;
  int64_t row0;
};

template <bool kWords>
__global__ __launch_bounds__(kStreamThreads, 2) void grouped_gemm_stream_kernel(Segments seg,
                                                                                GemmArgs ga) {
  __shared__ __align__(16) StreamShared sh;
  const int pieces = scalar(plan_segments<kStreamThreads>(seg, kStreamTokens, sh.plan, ga.status));
  const int lane = threadIdx.x & 63, wave = scalar(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int C = ga.C, G = C / kFp8Group, SG = kWords ? G / 4 : G;  // scale entries of a row
  const int nblk = (ga.N + kStreamN - 1) / kStreamN;
  // (at most a piece per expert and 2^15 blocks: 32 bits, also with a step on top)
  const uint32_t units = (uint32_t)pieces * nblk;
  if (units == 0) return;
  const bool split = units * 2 <= gridDim.x * kStreamWaves;  // uniform
  const uint32_t u_first = split ? blockIdx.x : blockIdx.x * kStreamWaves + wave;
  const uint32_t u_step = split ? gridDim.x : gridDim.x * kStreamWaves;
  const int g_first = split ? wave : 0, g_step = split ? kStreamWaves : 1;

  auto unit = [&](uint32_t u) {  // one piece per segment: its blocks of weight rows in turn
    StreamUnit x;
    x.e = scalar(plan_find(sh.plan, seg.E, (int)(u / nblk)));
    x.n0 = scalar((int)(u - (uint32_t)scalar(sh.plan.first[x.e]) * nblk)) * kStreamN;
    // (from LDS: a load from memory here would wait for every copy in flight)
    x.tokens = scalar(sh.plan.rows[x.e]);
    x.row0 = scalar(sh.plan.start[x.e]);
    return x;
  };

  // where the next copies come from
  const uint8_t *wbase = nullptr, *tbase = nullptr;
  uint32_t wo[kStreamN / 8], to[kStreamTokens / 8];
  const uint32_t *sp = nullptr;  // the lane's scale
  int64_t s_step = 0;            // to the next group's (words: next four groups')
  auto open = [&](uint32_t u) {
    const StreamUnit x = unit(u);
    wbase = scalar(ga.w + ((int64_t)x.e * ga.N + x.n0) * C);
    tbase = scalar(ga.a + x.row0 * C);
    const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
    for (int i = 0; i < kStreamN / 8; ++i)
      wo[i] = (uint32_t)min(i * 8 + (lane >> 3), ga.N - 1 - x.n0) * (uint32_t)C + chunk;
#pragma unroll
    for (int i = 0; i < kStreamTokens / 8; ++i)
      to[i] = (uint32_t)min(i * 8 + (lane >> 3), x.tokens - 1) * (uint32_t)C + chunk;
    if (lane < 16) {
      const int64_t r = x.row0 + min(lane, x.tokens - 1);
      const int64_t at = seg.per_expert > 0
                             ? (int64_t)x.e * SG * seg.per_expert +
                                   (r - (int64_t)x.e * seg.per_expert)
                             : r * SG;
      sp = static_cast<const uint32_t *>(ga.a_scale) + at;
      s_step = seg.per_expert > 0 ? seg.per_expert : 1;
    } else {
      sp = reinterpret_cast<const uint32_t *>(ga.w_scale) +
           ((int64_t)x.e * ((ga.N + 127) / 128) + x.n0 / 128) * G;
      s_step = 1;
    }
  };
  const uint32_t ring0 = lds_byte(sh.ring[wave]);
  auto issue = [&](int g, int slot) {
    const uint32_t st = ring0 + slot * (uint32_t)sizeof(StreamStage);
    const int64_t k = (int64_t)g * kFp8Group;
#pragma unroll
    for (int i = 0; i < kStreamN / 8; ++i) copy16_once(wbase + k, wo[i], st + i * 1024);
#pragma unroll
    for (int i = 0; i < kStreamTokens / 8; ++i)
      copy16_to_lds(tbase + k, to[i], st + kStreamN * 128 + i * 1024);
    copy4_to_lds_at(sp + (kWords && lane < 16 ? g >> 2 : g) * s_step,
                    st + (kStreamN + kStreamTokens) * 128);
  };

  f32x4 acc[2];
  auto multiply = [&](int g, const StreamStage &st) {
    const i32x8 a = rows16(st.a, 0);
    const float b = __uint_as_float(st.scale[16]);
    const float s = (kWords ? byte_scale(st.scale[l16], g & 3) : __uint_as_float(st.scale[l16])) * b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 m = mfma_group(rows16(st.w, i), a);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = __builtin_fmaf(m[c], s, acc[i][c]);
    }
  };

  uint32_t u_copy = u_first;  // next to copy: group g_copy of unit u_copy
  int g_copy = g_first, slot_copy = 0, ahead = 0;
  auto advance = [&]() {  // copies the next group, if there is one
    if (u_copy >= units) return;
    issue(g_copy, slot_copy);
    slot_copy = slot_copy == kStreamRing - 1 ? 0 : slot_copy + 1;
    ++ahead;
    g_copy += g_step;
    if (g_copy >= G) {
      g_copy = g_first;
      u_copy += u_step;
      if (!split && u_copy < units) open(u_copy);
    }
  };
  int slot = 0;
  for (uint32_t u = u_first; u < units; u += u_step) {
    acc[0] = acc[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (u == u_first || split) {
      open(u);
      u_copy = g_first < G ? u : units;
      g_copy = g_first;
      slot_copy = slot = ahead = 0;
      for (int i = 0; i < kStreamRing - 1; ++i)
        if (!split || u_copy == u) advance();
    }
    for (int g = g_first; g < G; g += g_step) {
      if (!split || u_copy == u) advance();
      // `ahead` groups are in flight or landed; the first of them is needed
      if (ahead == 3)
        __builtin_amdgcn_s_waitcnt(0x0f7e);  // vmcnt(14): two groups' copies may be out
      else if (ahead == 2)
        __builtin_amdgcn_s_waitcnt(0x0f77);  // vmcnt(7)
      else
        __builtin_amdgcn_s_waitcnt(0x0f70);
      asm volatile("" ::: "memory");
      multiply(g, sh.ring[wave][slot]);
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the slot is read, and free
      asm volatile("" ::: "memory");
      slot = slot == kStreamRing - 1 ? 0 : slot + 1;
      --ahead;
    }
    const StreamUnit x = unit(u);
    if (!split) {
      uint16_t *o = ga.out + (x.row0 + l16) * ga.N + x.n0 + quad * 4;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (l16 < x.tokens && x.n0 + i * 16 + quad * 4 < ga.N)
          *reinterpret_cast<ex_u32x2 *>(o + i * 16) =
              ex_u32x2{ex_bf16x2(acc[i][0], acc[i][1]), ex_bf16x2(acc[i][2], acc[i][3])};
      continue;
    }
    // the waves' sums, in the place of their rings (all copies have landed)
    float *part = reinterpret_cast<float *>(sh.ring[wave]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        part[l16 * (kStreamN + 1) + i * 16 + quad * 4 + c] = acc[i][c];
    __syncthreads();
    const int t = threadIdx.x >> 5, n = threadIdx.x & 31;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kStreamWaves; ++w)
      sum += reinterpret_cast<const float *>(sh.ring[w])[t * (kStreamN + 1) + n];
    if (t < x.tokens && x.n0 + n < ga.N)
      ga.out[(x.row0 + t) * ga.N + x.n0 + n] = (uint16_t)ex_bf16(sum);
    __syncthreads();
  }
}

// ---- tiles: segments of many rows -------------------------------------------
//
// A tile is 192 weight rows x up to 288 token rows. The larger the tile, the fewer
// bytes a product copies, and 288 rows are the most that fit: the float sums (3 x 9
// of 16 x 16 per wave) and operands fill the 256 registers of eight waves, the
// buffers LDS (four waves of 512 registers are not tried). At 8192 tokens x 8 over
// 256 experts, 7168 channels to 4096, most experts are one piece: 8.6 GB read, 8.0
// at least.
// What bounds it (that product: 2420 us, 1590 TFLOP/s): the copies without the
// products take 2230 us, the products without the copies 1670, all without memory
// (rows and weights from L2) 1965. The matrix units are busy 45% of the clocks, at
// 1.7 to 2.1 GHz: under this load the GPU's power holds the clock down, so that the
// products cost as much as the overlap would win. The skewed batch (4096 tokens
// x 6 over 64 experts, 4096 to 2824): 400 us, 1420 TFLOP/s, from pieces of 32 rows'
// steps and a last round of tiles that does not fill the chip.
// Tried and slower: 256 weight rows with two buffers (2884 us with the copies
// of that time); weights copied by four waves and rows by the others (+9%); the
// weights' buffer given back at a barrier of its own (+14%); the next tile's
// lines fetched into L2 ahead (+35%); raised priority around the products (+3%).

constexpr int kTileWaves = 8;      // 4 along the weight rows x 2 along the token rows
constexpr int kTileThreads = kTileWaves * 64;
constexpr int kWaveN = 48;         // weight rows of a wave: 3 operands of 16
constexpr int kTileN = 4 * kWaveN;  // weight rows of a tile
constexpr int kTileMost = 9;       // 16-row token tiles per wave
constexpr int kTileTokens = 2 * 16 * kTileMost;

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
// Scales are kept for four groups at a time, and copied a block of four ahead:
// the copies of one group's row-major scales touch a line per token, as many
// lines as its 128 channels (1594 against 1175 us for the token copies alone of
// 65536 rows, 7168 channels, 22 tiles wide).
enum ScaleLayout {
  kScaleWord,    // a UE8M0 word holds the token's four groups
  kScaleVector,  // row-major floats, four of a token in one 16-byte copy
  kScaleSingle,  // anything else: a copy per group
};
constexpr int kScaleTokens = (kTileTokens + 63) / 64 * 64;  // whole copies of 64
struct TileScales {
  float tokens[4 * kScaleTokens];  // kScaleVector: [token][4], else [group][token]
  float weights[64];              // [16 weight rows][4]
};
struct TileBuffers {
  uint8_t w[3][kTileN * 128];
  uint8_t a[2][kTileTokens * 128];
  TileScales scale[2];
};

template <int TT, ScaleLayout kScale>
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
  constexpr int kSlots = kCopies + 4;  // copies of a group: rows, weights, scales
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
  const uint32_t lds_w = lds_byte(lds.w) + wave * 1024, lds_a = lds_byte(lds.a) + wave * 1024;
  // The i-th of a wave's three copies of a group's weights, and of its kCopies
  // of the token rows.
  auto copy_weights = [&](int g, int to, int i) {
    copy16_to_lds(wbase + (int64_t)min(g, G - 1) * kFp8Group, wo[i],
                  lds_w + to * (kTileN * 128) + i * kTileWaves * 1024);
  };
  auto copy_rows = [&](int g, int to, int i) {
    if ((i + 1) * kTileWaves <= TT * 4 || i * kTileWaves + wave < TT * 4)
      copy16_to_lds(tbase + (int64_t)min(g, G - 1) * kFp8Group, to_off[i],
                    lds_a + to * (kTileTokens * 128) + i * kTileWaves * 1024);
  };
  // Scales: waves 0-4 copy those of 64 tokens each, wave 5
  // those of the weights, a lane one of the twelve 16-row blocks and a group.
  const uint32_t *sbase = scalar(static_cast<const uint32_t *>(ga.a_scale) + p.scale_base);
  const uint32_t so = (uint32_t)min(wave * 64 + lane, p.tokens - 1) * (uint32_t)p.r_stride * 4;
  const bool scopy = wave < (TT + 1) / 2;  // uniform
  const float *wsbase =
      scalar(ga.w_scale + ((int64_t)p.e * ((ga.N + 127) / 128) + p.n0 / 128) * G);
  const uint32_t wblock =
      (uint32_t)(min(p.n0 + min(lane >> 2, 11) * 16, ga.N - 1) / 128 - p.n0 / 128) * (uint32_t)G;
  const uint32_t lds_s = lds_byte(lds.scale[0].tokens), lds_ws = lds_byte(lds.scale[0].weights);
  // Part `part` of the scales of block b (groups 4 b ... 4 b + 3); the float
  // layouts without whole vectors take a part per group, the others part 0.
  // Returns whether this wave copied (uniform).
  auto copy_scales = [&](int b, int part) {
    const uint32_t to = (b & 1) * (uint32_t)sizeof(TileScales);
    if (wave == 5 && part == 0) {
      copy4_to_lds(wsbase, (wblock + (uint32_t)min(4 * b + (lane & 3), G - 1)) * 4, lds_ws + to);
      return true;
    }
    if (!scopy || (kScale != kScaleSingle && part > 0)) return false;
    if (kScale == kScaleVector)
      copy16_to_lds(sbase + 4 * min(b, G / 4 - 1), so, lds_s + to + wave * 1024);
    else if (kScale == kScaleWord)
      copy4_to_lds(sbase + min(b, G / 4 - 1) * p.g_stride, so, lds_s + to + wave * 256);
    else
      copy4_to_lds(sbase + min(4 * b + part, G - 1) * p.g_stride, so,
                   lds_s + to + (part * kScaleTokens + wave * 64) * 4);
    return true;
  };

  f32x4 acc[3][TT];
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // Product q = 3 t + i (token tile t, weight rows i) is issued while product
  // q - 2 is scaled and added. The empty asm orders the two: left alone, the
  // compiler issues all products first, and their results do not fit the
  // registers.
  auto compute = [&](int g, const uint8_t *sw, const uint8_t *sa, const TileScales &sc,
                     auto copy) {
    const uint8_t *wbuf = sw + wn * kWaveN * 128, *buf = sa + wt * TT * 2048;
    const int gi = g & 3;
    auto scale = [&](int t) {
      const int r = (wt * TT + t) * 16 + l16;
      if (kScale == kScaleVector) return sc.tokens[r * 4 + gi];
      if (kScale == kScaleSingle) return sc.tokens[gi * kScaleTokens + r];
      return byte_scale(__float_as_uint(sc.tokens[r]), gi);
    };
    i32x8 w[3], a[3];
    float b[3], s[TT];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      w[i] = rows16(wbuf, i);
      if (i < 2 && i < TT) a[i] = rows16(buf, i);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) b[i] = sc.weights[(wn * 3 + i) * 4 + gi];
#pragma unroll
    for (int t = 0; t < TT; ++t) s[t] = scale(t);
    f32x4 m[3];
#pragma unroll
    for (int q = 0; q < 3 * TT + 2; ++q) {
      const int t = q / 3, i = q % 3;
      if (q < 3 * TT) {
        if (i == 0 && t + 2 < TT) a[(t + 2) % 3] = rows16(buf, t + 2);
        if (i == 1) {  // two at a time, or what it takes
          constexpr int kPer = kSlots > 2 * TT ? (kSlots + TT - 1) / TT : 2;
#pragma unroll
          for (int c = t * kPer; c < (t + 1) * kPer && c < kSlots; ++c) copy(c);
        }
        if (q >= 3) {
          f32x4 &done = acc[i][t - 1];
          asm volatile("" : "+v"(a[t % 3]), "+v"(done));
        }
        m[i] = mfma_group(w[i], a[t % 3]);
      }
      if (q >= 2) {
        const int d = q - 2, dt = d / 3, di = d % 3;
        const float f = s[dt] * b[di];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[di][dt][c] = __builtin_fmaf(m[di][c], f, acc[di][dt][c]);
      }
    }
  };
  // While a group is computed, the next group's token rows, the weights of the
  // group after that and the scales four groups on are on their way. At its end
  // all copies but those last ones of the weights and scales have landed, for
  // every wave. Groups past the last are copied again, not used.
  // The copies are issued between the products: in one burst at the start they
  // would hold the waves up until the address unit has taken them all.
#pragma unroll
  for (int i = 0; i < 4; ++i) copy_scales(0, i);
#pragma unroll
  for (int i = 0; i < kCopies; ++i) copy_rows(0, 0, i);
#pragma unroll
  for (int i = 0; i < 6; ++i) copy_weights(i / 3, i / 3, i % 3);
  __builtin_amdgcn_s_waitcnt(0x0f73);  // vmcnt(3)
  lds_barrier();
  int w_now = 0, w_free = 2;
  for (int g = 0; g < G; ++g) {
    bool more = false;
    compute(g, lds.w[w_now], lds.a[g & 1], lds.scale[(g >> 2) & 1], [&](int c) {
      if (c < kCopies)
        copy_rows(g + 1, (g + 1) & 1, c);
      else if (c < kCopies + 3)
        copy_weights(g + 2, w_free, c - kCopies);
      else
        more = copy_scales((g >> 2) + 1, g & 3);
    });
    w_free = w_now;
    w_now = w_now == 2 ? 0 : w_now + 1;
    if (more)
      __builtin_amdgcn_s_waitcnt(0x0f74);  // vmcnt(4)
    else
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

template <ScaleLayout kScale>
__global__ __launch_bounds__(kTileThreads, 2) void grouped_gemm_tile_kernel(Segments seg,
                                                                            GemmArgs ga) {
  __shared__ SegmentPlan plan;
  __shared__ __align__(16) TileBuffers lds;
  const int pieces = scalar(plan_segments<kTileThreads>(seg, kTileTokens, plan, ga.status));
  const int G = ga.C / kFp8Group, SG = kScale == kScaleWord ? G / 4 : G;  // scale entries of a row
  const int nblk = (ga.N + kTileN - 1) / kTileN;
  // Workgroup b runs on XCD b % 8. In every round the XCD's workgroups take
  // neighbouring tiles, which share weights and token rows in its L2; the rounds
  // go through the experts together, so that one with many rows does not stay
  // with one XCD.
  // (32 bits: more tiles than that would have results past any memory)
  const uint32_t tiles = (uint32_t)pieces * nblk;
  const uint32_t lanes = gridDim.x >> 3;
  for (uint32_t u = (blockIdx.x & 7) * lanes + (blockIdx.x >> 3); u < tiles; u += gridDim.x) {
    TilePos p;
    // wave-uniform values, kept in scalar registers
    p.e = scalar(plan_find(plan, seg.E, (int)(u / nblk)));
    const int first = scalar(plan.first[p.e]), np = scalar(plan.first[p.e + 1]) - first;
    const int r = scalar((int)(u - (uint32_t)first * nblk));
    const int nb = scalar(r / np), piece = r - nb * np;
    const int count = scalar(seg.count[p.e]);
    const int per = scalar(((count + np - 1) / np + 31) & ~31);  // the pieces are even
    p.tokens = min(count - piece * per, per);
    p.row0 = (int64_t)scalar(seg.start[p.e]) + piece * per;
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
      case 1: case 2: tile_product<2, kScale>(ga, p, lds); break;
      case 3: tile_product<3, kScale>(ga, p, lds); break;
      case 4: tile_product<4, kScale>(ga, p, lds); break;
      case 5: tile_product<5, kScale>(ga, p, lds); break;
      case 6: tile_product<6, kScale>(ga, p, lds); break;
      case 7: tile_product<7, kScale>(ga, p, lds); break;
      case 8: tile_product<8, kScale>(ga, p, lds); break;
      default: tile_product<9, kScale>(ga, p, lds); break;
    }
  }
}

// A segment of one stream unit's rows is streamed, a larger one tiled. (With
// the border at 32 or 64 rows, streamed in pieces of 16 that read the weights
// again: 1024 x 8 rows over 256 experts, 7168 x 4096, 4.3 or 3.0 TB/s of weights
// against 5.4; 128 x 8 rows over 32 experts 3.3 or 3.1 against 4.8.)
constexpr int kStreamMost = kStreamTokens;

}  // namespace

hipError_t launch_grouped_gemm(const Segments &seg, const GemmArgs &g, hipStream_t s) {
  const bool words = g.flags & kFp8Ue8m0;
  const int64_t nblk = (g.N + kStreamN - 1) / kStreamN;
  const int64_t most = seg.E * nblk;
  const unsigned grid = (unsigned)(most < 256 ? most : 256);  // one workgroup per CU
  // how many rows a segment can have at most decides which kernels are needed
  const int64_t bound = seg.max_count > 0 ? seg.max_count
                                          : (seg.per_expert > 0 ? seg.per_expert : seg.rows);
  Segments part = seg;
  part.upto = kStreamMost;
  if (words)
    hipLaunchKernelGGL((grouped_gemm_stream_kernel<true>), dim3(grid), dim3(kStreamThreads), 0, s,
                       part, g);
  else
    hipLaunchKernelGGL((grouped_gemm_stream_kernel<false>), dim3(grid), dim3(kStreamThreads), 0, s,
                       part, g);
  if (bound > kStreamMost) {
    part.over = kStreamMost;
    part.upto = 0;
    // row-major float scales in whole 16-byte vectors: every row starts on one
    const bool vectors = seg.per_expert == 0 && (g.C / kFp8Group) % 4 == 0 &&
                         (reinterpret_cast<uintptr_t>(g.a_scale) & 15u) == 0;
    if (words)
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<kScaleWord>), dim3(256), dim3(kTileThreads), 0,
                         s, part, g);
    else if (vectors)
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<kScaleVector>), dim3(256), dim3(kTileThreads), 0,
                         s, part, g);
    else
      hipLaunchKernelGGL((grouped_gemm_tile_kernel<kScaleSingle>), dim3(256), dim3(kTileThreads), 0,
                         s, part, g);
  }
  return hipGetLastError();
}

}  // namespace moe
