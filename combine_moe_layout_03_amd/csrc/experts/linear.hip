// Dense product of bf16 rows with bias, activation and residual in its
// epilogue, and the products of its gradients:
//   out[t][n] = act( sum_c x[t][c] w[n][c] + bias[n] ) + residual[t][n]
//   d_x[t][c] = sum_n d_z[t][n] w[n][c],   d_w[n][c] = sum_t d_z[t][n] x[t][c]
//
// All three are D[r][c] = sum_k R(r, k) C(c, k) with an operand stored either
// along k ([r][k]) or across it ([k][r]); only the copies to LDS and the reads of
// the fragments differ. The columns' operand comes first in the matrix
// instruction (16 x 16 x 32), so that a lane's four results are neighbours in a
// row of D. Sums are float: those of 7168 products are off by 5e-7 of the result's norm
// (a chain of fused multiply-adds by 9e-7).
#include "linear.hpp"
#include "linear_plan.hpp"

#include <utility>

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// s_waitcnt's operand: at most n vector memory operations still out.
constexpr int vmcnt(int n) { return 0x0f70 | (n & 15) | (n >> 4) << 14; }

// f(0), f(1), ..., f(kN - 1), each number a type of its own.
template <class F, int... kI>
__device__ __forceinline__ void each_of(F &f, std::integer_sequence<int, kI...>) {
  (f(std::integral_constant<int, kI>{}), ...);
}
template <int kN, class F>
__device__ __forceinline__ void each(F f) {
  each_of(f, std::make_integer_sequence<int, kN>{});
}

struct ProductArgs {
  const uint16_t *r, *c;
  int32_t rows, cols, k;  // of D; of the sum
  int32_t r_ld, c_ld;     // elements of an operand's row in memory
  int32_t col_units;      // tiles along the columns
  int32_t splits;         // parts of k; more than one: partial sums to ws[part][rows][ws_cols]
  int32_t split_steps;    // stages of a part
  float *ws;
  LinearEpilogue e;
};

// ---- tiles --------------------------------------------------------------------
//
// Four waves share a tile of up to 256 x 256, one wave a SIMD: each has 128 x 128 sums
// in its 256 accumulation registers and a whole stage's fragments, in two halves, in
// the others. So a stage's 64 KB are read from LDS once per two waves (1024 of the 2048
// clocks that its products take; with eight waves of 128 x 64 it would be 1536), and
// LDS is free for the stage after next as soon as the second half is in registers.
//
// What bounds it: 8192 x 4096 x 7168 take 314 to 353 us on different GPUs of this kind
// (1360 to 1530 TFLOP/s; a library product of this size 294 to 319), the gradients 347
// to 390 both (362 to 395, 488): the matrix units are busy 60% of the clocks at 1.9 GHz,
// where the GPU's power holds them. About 9 us go around every tile: its start, and its
// sums on their way out. 8192 x 7168 x 2048 186 to 209 us, with bias and residual 214 to
// 232 (the library 171 to 188 without); SwiGLU of 8192 x 2 x 2048 x 7168 338 to 356, with
// z kept 344 to 365.
// Measured and not kept (us, beside the kernel of that time): copies issued in one
// half of a stage for the next one 364 against 346; reads and copies in clumps before
// every eight products 351 against 338; tiles taken in turn by resident workgroups that
// start the next one's copies before they store 203 against 198; panels of 2, 6 or 8
// tiles, other places for the two barriers: within 2%; products of 32 x 32 x 16 360
// against 337; sums stored past L2 1% less for bf16 and 2 to 10% more for float.
//
// An operand stage in LDS. Along k: rows of 128 bytes, the 16-byte chunk c of
// row r at chunk c ^ (r & 7). Across k: 64 rows (k) of the tile's width, the
// 32-byte chunk m of row k at m ^ spread(k), where spread puts the eight rows that
// 32 lanes of a transposing read touch on all banks.
__device__ __forceinline__ int spread(int k) { return (k & 3) | ((k >> 1) & 4); }

constexpr int stage_rows(int rows, bool across) {
  return !across ? rows : rows > 128 ? 256 : 128;
}

struct Stage {
  ex_i32x4 buf;
  uint32_t to;
};

// How a wave copies its part of an operand's stages: kN copies a stage.
template <int kRows, int kWaves, bool kAcross, bool kPairs>
struct StageCopy {
  // (across k a row of the buffer is a power of two wide; what is over is not used)
  static constexpr int kWide = stage_rows(kRows, kAcross), kN = kWide / 8 / kWaves;
  uint64_t base;  // the tile's first element at the part's first k
  int64_t left;   // bytes from there to the operand's end
  uint32_t step;  // bytes to the next stage
  uint32_t off[kN];
  int lane_k;  // along k: the lane's first channel in a stage
  uint32_t lds;

  // row0: the tile's first row; with kPairs (SwiGLU weights) rows are taken in
  // blocks of 16, in turn from the first and from the second half of 2 * half rows.
  __device__ __forceinline__ void init(const uint16_t *p, int row0, int64_t rows, int ld, int k,
                                       int k0, const void *to, int half) {
    const int lane = threadIdx.x & 63, wave = scalar_i(threadIdx.x >> 6);
    lds = lds_offset(to) + wave * 1024;
    const int64_t bytes = (kAcross ? (int64_t)k : rows) * ld * 2;
    int64_t first;
    if (kAcross) {
      constexpr int kRowBytes = kWide * 2, kPer = 1024 / kRowBytes;
      first = ((int64_t)k0 * ld + row0) * 2;
      step = (uint32_t)ld * 2 * kStep;
      lane_k = 0;
      const int in = lane * 16 % kRowBytes;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int kr = (i * kWaves + wave) * kPer + lane * 16 / kRowBytes;
        off[i] = (uint32_t)kr * (uint32_t)ld * 2 + (((in >> 5) ^ spread(kr)) << 5 | (in & 16));
      }
    } else {
      const int chunk = (lane & 7) ^ (lane >> 3);
      lane_k = chunk * 8;
      step = kStep * 2;
      int shift = row0;
      if (kPairs) shift = row0 / 2 + (wave >> 1 & 1) * half;  // a wave copies from one half
      first = ((int64_t)shift * ld + k0) * 2;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        int r = (i * kWaves + wave) * 8 + (lane >> 3);
        if (kPairs) r = (r >> 5) * 16 + (r & 15);
        off[i] = (uint32_t)r * (uint32_t)ld * 2 + chunk * 16;
      }
    }
    base = scalar_u64((uint64_t)(uintptr_t)p + first);
    left = (int64_t)scalar_u64((uint64_t)(bytes - first));
  }
  // Stage s; nothing of it is read if it is off.
  __device__ __forceinline__ Stage stage(int s, bool on) const {
    const uint64_t at = (uint64_t)s * step;
    return {buffer_at(base + at, on ? left - (int64_t)at : 0), lds + (s & 1) * (kWide * 128)};
  }
  // Before the copies of a stage in which only `rest` channels are left, the last:
  // along k, chunks past them become zeros.
  __device__ __forceinline__ void cut(int rest) {
    if (kAcross) return;
#pragma unroll
    for (int i = 0; i < kN; ++i) off[i] = lane_k >= rest ? kOutside : off[i];
  }
  template <int kI>
  __device__ __forceinline__ void copy(const Stage &g) const {
    copy16_bounded<kI * kWaves * 1024>(g.buf, off[kI], g.to);
  }
};

// Fragment t (16 rows from row t * 16), channels 32 kk ... + 31 of a stage.
template <int kRows, bool kAcross>
__device__ __forceinline__ bf16x8 fragment(const uint8_t *stage, int t, int kk) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
  if (kAcross) {
    constexpr int kRowBytes = stage_rows(kRows, true) * 2;
    const int kr = kk * 32 + quad * 8 + (l16 >> 2);
    const int at = kr * kRowBytes + ((t ^ spread(kr)) << 5) + (l16 & 3) * 8;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(stage + at));
    const s16x4 b =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(stage + at + 4 * kRowBytes));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    const int at = t * 2048 + l16 * 128 + (((kk * 4 + quad) ^ (l16 & 7)) * 16);
    return *reinterpret_cast<const bf16x8 *>(stage + at);
  }
}

// acc += C R^T of 16 x 16 x 32. In asm, because the compiler, left to place 512
// registers, moves sums and fragments to and fro between the two files (dw of 8192 x
// 4096 x 7168: 461 us, with the sums held in the accumulation registers 389). It
// still waits for the fragments it reads; that the sums are ready, products_done()
// sees to (a product takes 16 clocks). Nothing in the source keeps a copy
// of a sum from being placed ahead of its waits: as operands of the waits the sums are
// copied, in part before them (204 us against 202 at 8192 x 7168 x 2048). So a test reads
// the built code: no result read, and no operand written, within the wait states.
__device__ __forceinline__ void product(f32x4 &acc, bf16x8 c, bf16x8 r) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(c), "v"(r));
}
__device__ __forceinline__ void products_done() {
  asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15" ::: "memory");
}

// 2 x 2 waves, each with kRT x kCT fragments of 16.
template <int kRT, int kCT, bool kRAcross, bool kCAcross, int kAct>
__global__ __launch_bounds__(256, kRT * kCT > 32 ? 1 : 2) void product_kernel(ProductArgs a) {
  constexpr int kRW = 2, kCW = 2;
  constexpr int kWaves = kRW * kCW, kR = kRW * kRT * 16, kC = kCW * kCT * 16;
  constexpr bool kPairs = kAct == kActSwiglu;
  constexpr int kRBytes = stage_rows(kR, kRAcross) * 128, kCBytes = stage_rows(kC, kCAcross) * 128;
  __shared__ __align__(1024) uint8_t lds[2 * (kRBytes + kCBytes)];
  uint8_t *const lds_r = lds, *const lds_c = lds + 2 * kRBytes;
  // Workgroup b runs on XCD b % 8: every XCD takes a run of neighbouring tiles,
  // four tiles high, which share operands in its L2.
  const int row_units = (a.rows + kR - 1) / kR, tiles = row_units * a.col_units;
  const int units = tiles * a.splits, per = (units + 7) / 8;
  const int u = scalar_i((int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3));
  if ((int)(blockIdx.x >> 3) >= per || u >= units) return;
  const int part = scalar_i((uint32_t)u / (uint32_t)tiles), tile = u - part * tiles;
  constexpr int kHigh = 4;
  const int panel = scalar_i((uint32_t)tile / (uint32_t)(kHigh * a.col_units));
  const int in = tile - panel * kHigh * a.col_units;
  const int high = min(kHigh, row_units - panel * kHigh);
  const int cu = scalar_i((uint32_t)in / (uint32_t)high);
  const int row0 = (panel * kHigh + in - cu * high) * kR, col0 = cu * kC;

  const int lane = threadIdx.x & 63, wave = scalar_i(threadIdx.x >> 6);
  const int wr = wave / kCW, wc = wave % kCW;
  const int k0 = part * a.split_steps * kStep;
  const int left = (a.k - k0 + kStep - 1) / kStep;
  const int n = min(left, a.split_steps);

  StageCopy<kR, kWaves, kRAcross, false> cr;
  StageCopy<kC, kWaves, kCAcross, kPairs> cc;
  cr.init(a.r, row0, a.rows, a.r_ld, a.k, k0, lds_r, 0);
  cc.init(a.c, col0, kPairs ? 2 * (int64_t)a.e.N : a.cols, a.c_ld, a.k, k0, lds_c, a.e.N);
  constexpr int kRN = decltype(cr)::kN, kCN = decltype(cc)::kN;
  f32x4 acc[kRT][kCT];
#pragma unroll
  for (int i = 0; i < kRT; ++i)
#pragma unroll
    for (int j = 0; j < kCT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // A stage is 2 kRT kCT products: first those of its channels 0-31, whose
  // fragments were read during the stage before, then those of 32-63, read behind
  // the first products. From product kFree on, behind a barrier, the stage's LDS is
  // free, and the copies of the stage after next go there: they have more than a
  // stage's time to land. From kNext on, behind another barrier, the next stage has
  // landed and its first fragments are read. A wave has its SIMD to itself and
  // issues about three instructions while a product runs, so reads and copies stand
  // one by one between the products.
  constexpr int kItems = kRT + kCT, kCopies = kRN + kCN, kTotal = 2 * kRT * kCT;
  constexpr int kFree = kTotal * 3 / 8, kNext = kTotal * 3 / 4;
  constexpr int kReadEvery = kFree * 5 / 6 / kItems;
  constexpr int kNextEvery =
      (kTotal - kNext) / kItems < 2 ? 1 : (kTotal - kNext) * 3 / 4 / kItems;
  constexpr int kCopyEvery = (kTotal - kFree) / kCopies;
  static_assert(kReadEvery > 0 && kNextEvery > 0 && kCopyEvery > 0, "a place for each");
  constexpr int kEarly = (kNext - kFree + kCopyEvery - 1) / kCopyEvery;
  constexpr int kAhead = kEarly < kCopies ? kEarly : kCopies;
  bf16x8 fr[2][kRT], fc[2][kCT];
  // item m: the columns' fragments 0 ... kCT - 1, then the rows'
  auto read = [&](int s, int kk, int m) {
    if (m < kCT)
      fc[kk][m] = fragment<kC, kCAcross>(lds_c + (s & 1) * kCBytes, wc * kCT + m, kk);
    else
      fr[kk][m - kCT] = fragment<kR, kRAcross>(lds_r + (s & 1) * kRBytes, wr * kRT + m - kCT, kk);
  };
  auto copy = [&](const Stage &gr, const Stage &gc, auto i) {
    if constexpr (i.value < kRN)
      cr.template copy<i.value>(gr);
    else
      cc.template copy<i.value - kRN>(gc);
  };
  const int rest = a.k - k0 - (n - 1) * kStep;  // channels of the last stage, or more
  auto cut_at = [&](int s) {
    if (s == n - 1 && rest < kStep) {
      cr.cut(rest);
      cc.cut(rest);
    }
  };

  for (int s = 0; s < 2; ++s) {
    cut_at(s);
    const Stage gr = cr.stage(s, s < n), gc = cc.stage(s, s < n);
    each<kCopies>([&](auto i) { copy(gr, gc, i); });
  }
  __builtin_amdgcn_s_waitcnt(vmcnt(kCopies));
  lds_barrier();
#pragma unroll
  for (int m = 0; m < kItems; ++m) read(0, 0, m);
  for (int s = 0; s < n; ++s) {
    Stage gr, gc;
    each<kTotal>([&](auto at) {
      constexpr int p = at.value, kk = p / (kRT * kCT), i = p / kCT % kRT, j = p % kCT;
      if constexpr (p == kFree) {
        lds_barrier();
        cut_at(s + 2);
      }
      if constexpr (p == kNext) {
        __builtin_amdgcn_s_waitcnt(vmcnt(kAhead));
        lds_barrier();
      }
      product(acc[i][j], fc[kk][j], fr[kk][i]);
      if constexpr (p % kReadEvery == 0 && p / kReadEvery < kItems) read(s, 1, p / kReadEvery);
      if constexpr (p == kFree / 2) gr = cr.stage(s + 2, s + 2 < n);
      if constexpr (p == kFree * 3 / 4) gc = cc.stage(s + 2, s + 2 < n);
      if constexpr (p >= kFree && (p - kFree) % kCopyEvery == 0 && (p - kFree) / kCopyEvery < kCopies)
        copy(gr, gc, std::integral_constant<int, (p - kFree) / kCopyEvery>{});
      if constexpr (p >= kNext && (p - kNext) % kNextEvery == 0 && (p - kNext) / kNextEvery < kItems)
        read(s + 1, 0, (p - kNext) / kNextEvery);
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  __builtin_amdgcn_s_waitcnt(vmcnt(0));  // no copy outlives the workgroup
  products_done();

  // The sums go through LDS, 32 rows of a wave at a time, so that a lane finishes eight
  // neighbouring columns: whole lines of the output and the residual.
  lds_barrier();  // no wave reads its stages any more
  const int l16 = lane & 15, quad = lane >> 4;
  constexpr int kPitch = kCT * 64 + 16;                   // bytes of a row: all banks in turn
  constexpr int kPer = kCT * 2 / (kPairs ? 2 : 1);        // lanes of a row
  constexpr int kPasses = kPer / 2;
  static_assert(4 * 32 * kPitch <= sizeof(lds), "the rows fit");
  uint8_t *const mine = lds + wave * (32 * kPitch);
  const int n0 = (col0 + wc * kCT * 16) / (kPairs ? 2 : 1);
  auto row = [&](int p) { return (p * 64 + lane) / kPer; };
  auto col = [&](int p) { return (p * 64 + lane) % kPer * 8; };  // of the wave's
  ex_u32x4 res[kRT / 2][kPasses];  // all of the residual at once: one wait for memory
  if (a.splits == 1 && a.e.residual) {
#pragma unroll
    for (int i = 0; i < kRT / 2; ++i)
#pragma unroll
      for (int p = 0; p < kPasses; ++p)
        res[i][p] = linear_residual(
            a.e, min(row0 + (wr * kRT + 2 * i) * 16 + (int64_t)row(p), (int64_t)a.rows - 1),
            min(n0 + col(p), a.e.N - 8));
  }
  each<kRT / 2>([&](auto pair) {
    constexpr int i = 2 * pair.value;
    const int64_t t0 = row0 + (wr * kRT + i) * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < kCT; ++j)
        *reinterpret_cast<f32x4 *>(mine + (h * 16 + l16) * kPitch + j * 64 + quad * 16) =
            acc[i + h][j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    f32x8 zs[kPasses], ups[kPairs ? kPasses : 1];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      // a pair's blocks of 16 stand next to each other
      const int c = kPairs ? (col(p) & ~15) * 2 + (col(p) & 15) : col(p);
      const float *from = reinterpret_cast<const float *>(mine + row(p) * kPitch) + c;
      zs[p] = two_of(from);
      if (kPairs) ups[p] = two_of(from + 16);
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const f32x8 z = zs[p], up = kPairs ? ups[p] : z;
      const int64_t t = t0 + row(p);
      const int n = n0 + col(p);
      if (t >= a.rows || n >= a.e.N) continue;
      if (a.splits > 1) {  // as they are
        const int64_t NN = kPairs ? 2 * (int64_t)a.e.N : a.e.N;
        float *o = a.ws + ((int64_t)part * a.rows + t) * NN + n;
        *reinterpret_cast<f32x4 *>(o) = f32x4{z[0], z[1], z[2], z[3]};
        *reinterpret_cast<f32x4 *>(o + 4) = f32x4{z[4], z[5], z[6], z[7]};
        if (kPairs) {
          *reinterpret_cast<f32x4 *>(o + a.e.N) = f32x4{up[0], up[1], up[2], up[3]};
          *reinterpret_cast<f32x4 *>(o + a.e.N + 4) = f32x4{up[4], up[5], up[6], up[7]};
        }
      } else {
        linear_store<kAct>(a.e, t, n, z, up, res[pair.value][p]);
      }
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_sched_barrier(0);
  });
}

// Adds the parts of a split product up, in order, and finishes them.
template <int kAct>
__global__ __launch_bounds__(256) void join_kernel(ProductArgs a) {
  constexpr bool kPairs = kAct == kActSwiglu;
  const int NN = kPairs ? 2 * a.e.N : a.e.N, per = a.e.N / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.rows * per) return;
  const int64_t t = i / per;
  const int n = (int)(i - t * per) * 8;
  const float *p = a.ws + t * NN + n;
  const int64_t part = (int64_t)a.rows * NN;
  const ex_u32x4 res = linear_residual(a.e, t, n);
  f32x8 z = two_of(p), up = z;
  if (kPairs) up = two_of(p + a.e.N);
  for (int s = 1; s < a.splits; ++s) {
    p += part;
    z += two_of(p);
    if (kPairs) up += two_of(p + a.e.N);
  }
  linear_store<kAct>(a.e, t, n, z, up, res);
}

// ---- stream: few rows -----------------------------------------------------------
//
// Few rows make this a read of the weights. A workgroup takes kW rows of them (SwiGLU:
// half of them gates) and 16 tokens; its waves share the channels out in groups of
// 64, each through a ring of groups in its own part of LDS, without a barrier, and
// join their sums at the end.
//
// 16 tokens, 7168 to 4096 channels, weights from memory: 12.1 us, 4.9 TB/s of them (they
// come through L2 beside as many bytes of tokens); 128 tokens, 7168 to 256: 6.5 us (13.4
// as split tiles), about 38 bytes a clock into a CU; what bounds it is that each block of
// 16 tokens brings the weights in again, 88 MB in all for 5.5. Rings of 2, 3, 4 or 8 groups
// and 4, 8 or 16 waves: within 5%, but for those that leave a CU one workgroup, slower
// where there are more.

constexpr int kStreamWaves = 4, kStreamRing = 4;

template <int kW, int kAct>
__global__ __launch_bounds__(kStreamWaves * 64) void stream_kernel(ProductArgs a) {
  constexpr bool kPairs = kAct == kActSwiglu;
  constexpr int kOut = kPairs ? kW / 2 : kW, kCopies = 2 + kW / 8, kRows = 16 + kW;
  constexpr int kPitch = 20;  // floats of a token's sums
  // (with kW = 8 the instruction's other weight rows are what stands behind the group)
  __shared__ __align__(1024) uint8_t ring[kStreamWaves * kStreamRing * kRows * 128 + 1024];
  static_assert(16 * kPitch * 4 <= kStreamRing * kRows * 128, "sums replace a wave's ring");
  const int lane = threadIdx.x & 63, wave = scalar_i(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  // Workgroup b runs on XCD b % 8: an XCD takes neighbouring weight rows for all tokens,
  // so that its L2 holds an eighth of the weights.
  const int blocks = (a.rows + 15) / 16, units = a.col_units * blocks, per = (units + 7) / 8;
  const int u = scalar_i((int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3));
  if ((int)(blockIdx.x >> 3) >= per || u >= units) return;
  const int nb = scalar_i((uint32_t)u / (uint32_t)blocks);
  const int n0 = nb * kOut, t0 = (u - nb * blocks) * 16;
  const int64_t ld = (int64_t)a.c_ld * 2;  // bytes of a row, of both operands
  const ex_i32x4 wbuf = buffer_at(scalar_u64((uint64_t)(uintptr_t)a.c + n0 * ld),
                                  (int64_t)scalar_u64((uint64_t)((a.cols - n0) * ld)));
  const ex_i32x4 tbuf = buffer_at(scalar_u64((uint64_t)(uintptr_t)a.r + t0 * ld),
                                  (int64_t)scalar_u64((uint64_t)((a.rows - t0) * ld)));
  const int chunk = (lane & 7) ^ (lane >> 3), row = lane >> 3;
  uint32_t w_off[kW / 8], t_off[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = i * 8 + row;
    t_off[i] = (uint32_t)r * (uint32_t)ld + chunk * 16;
    if (i < kW / 8)
      w_off[i] = (uint32_t)(kPairs && r >= kOut ? a.e.N + r - kOut : r) * (uint32_t)ld + chunk * 16;
  }
  const int groups = (a.k + kStep - 1) / kStep;
  uint8_t *const mine = ring + wave * (kStreamRing * kRows * 128);
  const uint32_t lds = lds_offset(mine);
  auto issue = [&](int g, int slot) {  // groups past the last, and chunks, arrive as zeros
    const uint32_t more = (uint32_t)g * 128, mask = g * kStep + chunk * 8 < a.k ? 0u : kOutside;
    const uint32_t to = lds + slot * (kRows * 128);
#pragma unroll
    for (int i = 0; i < 2; ++i) copy16_bounded(tbuf, (t_off[i] + more) | mask, to + i * 1024);
#pragma unroll
    for (int i = 0; i < kW / 8; ++i) {
      if (blocks == 1)  // unmarked 8% more (16 x 4096 of 7168 channels)
        copy16_bounded_once(wbuf, (w_off[i] + more) | mask, to + 2048 + i * 1024);
      else  // the other tokens' workgroups read them too (marked 13% more, 128 x 256)
        copy16_bounded(wbuf, (w_off[i] + more) | mask, to + 2048 + i * 1024);
    }
  };
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kStreamRing - 1; ++i) issue(wave + i * kStreamWaves, i);
  int slot = 0;
  for (int g = wave; g < groups; g += kStreamWaves) {
    issue(g + (kStreamRing - 1) * kStreamWaves, (slot + kStreamRing - 1) % kStreamRing);
    __builtin_amdgcn_s_waitcnt(vmcnt((kStreamRing - 1) * kCopies));
    asm volatile("" ::: "memory");
    const uint8_t *st = mine + slot * (kRows * 128);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fragment<16, false>(st, 1, kk),
                                                    fragment<16, false>(st, 0, kk), acc, 0, 0, 0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the slot is read, and free
    asm volatile("" ::: "memory");
    slot = (slot + 1) % kStreamRing;
  }
  __builtin_amdgcn_s_waitcnt(vmcnt(0));  // also the zeros have landed
  lds_barrier();                         // and with kW = 8 a ring is read up into the next
  *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(mine) + l16 * kPitch + quad * 4) = acc;
  lds_barrier();
  constexpr int kPer = kOut / 4;  // threads of a token, four columns each
  if (threadIdx.x >= 16 * kPer) return;
  const int t = threadIdx.x / kPer, n = threadIdx.x % kPer * 4;
  f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f}, up = z;
#pragma unroll
  for (int w = 0; w < kStreamWaves; ++w) {
    const float *p =
        reinterpret_cast<const float *>(ring + w * (kStreamRing * kRows * 128)) + t * kPitch + n;
    z += *reinterpret_cast<const f32x4 *>(p);
    if (kPairs) up += *reinterpret_cast<const f32x4 *>(p + kOut);
  }
  if (t0 + t < a.rows && n0 + n < a.e.N) linear_store4<kAct>(a.e, t0 + t, n0 + n, z, up);
}

template <int kW, int kAct>
hipError_t launch_stream(ProductArgs a, hipStream_t s) {
  constexpr int kOut = kAct == kActSwiglu ? kW / 2 : kW;
  a.cols = kAct == kActSwiglu ? 2 * a.e.N : a.e.N;
  a.col_units = (a.e.N + kOut - 1) / kOut;
  hipLaunchKernelGGL((stream_kernel<kW, kAct>),
                     dim3((unsigned)((a.col_units * ((a.rows + 15) / 16) + 7) / 8 * 8)),
                     dim3(kStreamWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int kAct>
hipError_t launch_streamed(const ProductArgs &a, hipStream_t s) {
  return stream_weight_rows(a.rows, a.e.N, kAct == kActSwiglu) == 8 ? launch_stream<8, kAct>(a, s)
                                                                    : launch_stream<16, kAct>(a, s);
}

template <bool kRAcross, bool kCAcross, int kAct>
hipError_t launch_product(ProductArgs a, hipStream_t s) {
  const int64_t cols = kAct == kActSwiglu ? 2 * (int64_t)a.e.N : a.e.N;
  a.cols = (int32_t)cols;
  const Plan p = plan(a.rows, cols, a.k, kAct == kActSwiglu, kMaxWorkspace);
  a.col_units = (int32_t)((cols + 32 * p.wide - 1) / (32 * p.wide));
  a.splits = p.splits;
  a.split_steps = p.steps;
  const int64_t units = (int64_t)a.col_units * ((a.rows + 32 * p.high - 1) / (32 * p.high)) * p.splits;
  const dim3 grid((unsigned)((units + 7) / 8 * 8)), block(256);
  if (p.high == 4)
    hipLaunchKernelGGL((product_kernel<4, 4, kRAcross, kCAcross, kAct>), grid, block, 0, s, a);
  else if (p.wide == 8)
    hipLaunchKernelGGL((product_kernel<8, 8, kRAcross, kCAcross, kAct>), grid, block, 0, s, a);
  else if (p.wide == 7) {
    if constexpr (kAct != kActSwiglu)
      hipLaunchKernelGGL((product_kernel<8, 7, kRAcross, kCAcross, kAct>), grid, block, 0, s, a);
  } else
    hipLaunchKernelGGL((product_kernel<8, 6, kRAcross, kCAcross, kAct>), grid, block, 0, s, a);
  if (p.splits > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(join_kernel<kAct>,
                       dim3((unsigned)(((int64_t)a.rows * (a.e.N / 8) + 255) / 256)), dim3(256), 0,
                       s, a);
  }
  return hipGetLastError();
}

size_t plan_bytes(int64_t rows, int64_t cols, int64_t k, bool pairs = false) {
  if (rows == 0) return 0;
  const Plan p = plan(rows, cols, k, pairs, kMaxWorkspace);
  return p.splits > 1 ? (size_t)(p.splits * rows * cols * 4) : 0;
}

}  // namespace

size_t linear_workspace(int32_t T, int32_t N, int32_t C, int32_t act) {
  const bool pairs = act == kActSwiglu;
  if (streamed(T, N, C, pairs)) return 0;
  return plan_bytes(T, pairs ? 2 * (int64_t)N : N, C, pairs);
}
size_t linear_grad_workspace(int32_t T, int32_t N, int32_t C) {
  const size_t x = plan_bytes(T, C, N), w = plan_bytes(N, C, T);
  return x > w ? x : w;
}

hipError_t launch_linear(int32_t T, int32_t N, int32_t C, const uint16_t *x, const uint16_t *w,
                         const float *bias, const uint16_t *residual, void *out, uint16_t *pre,
                         int32_t act, bool f32, float *ws, hipStream_t s) {
  ProductArgs a{x, w, T, 0, C, C, C, 0, 1, 0, ws, {bias, residual, out, pre, N, f32}};
  if (streamed(T, N, C, act == kActSwiglu)) {
    switch (act) {
      case kActNone: return launch_streamed<kActNone>(a, s);
      case kActSilu: return launch_streamed<kActSilu>(a, s);
      case kActGelu: return launch_streamed<kActGelu>(a, s);
      default: return launch_streamed<kActSwiglu>(a, s);
    }
  }
  switch (act) {
    case kActNone: return launch_product<false, false, kActNone>(a, s);
    case kActSilu: return launch_product<false, false, kActSilu>(a, s);
    case kActGelu: return launch_product<false, false, kActGelu>(a, s);
    default: return launch_product<false, false, kActSwiglu>(a, s);
  }
}

hipError_t launch_linear_grad_x(int32_t T, int32_t N, int32_t C, const uint16_t *d_z,
                                const uint16_t *w, uint16_t *d_x, float *ws, hipStream_t s) {
  ProductArgs a{d_z, w, T, 0, N, N, C, 0, 1, 0, ws, {nullptr, nullptr, d_x, nullptr, C, false}};
  return launch_product<false, true, kActNone>(a, s);
}

hipError_t launch_linear_grad_w(int32_t T, int32_t N, int32_t C, const uint16_t *d_z,
                                const uint16_t *x, float *d_w, float *ws, hipStream_t s) {
  ProductArgs a{d_z, x, N, 0, T, N, C, 0, 1, 0, ws, {nullptr, nullptr, d_w, nullptr, C, true}};
  return launch_product<true, true, kActNone>(a, s);
}

}  // namespace moe
