// Dense product of bf16 rows with bias, activation and residual in its
// epilogue, and the products of its gradients:
//   out[t][n] = act( sum_c x[t][c] w[n][c] + bias[n] ) + residual[t][n]
//   d_x[t][c] = sum_n d_z[t][n] w[n][c],   d_w[n][c] = sum_t d_z[t][n] x[t][c]
//
// All three are D[r][c] = sum_k R(r, k) C(c, k) with an operand stored either
// along k ([r][k]) or across it ([k][r]); only the copies to LDS and the reads of
// the fragments differ. The columns' operand comes first in the matrix
// instruction (16 x 16 x 32), so that a lane's four results are neighbours in a
// row of D. Sums are float.
#include "linear.hpp"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// s_waitcnt's operand: at most n vector memory operations still out.
constexpr int vmcnt(int n) { return 0x0f70 | (n & 15) | (n >> 4) << 14; }

constexpr int kStep = 64;  // k of a stage: 128 bytes of a row

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
// An operand stage in LDS. Along k: rows of 128 bytes, the 16-byte chunk c of
// row r at chunk c ^ (r & 7). Across k: 64 rows (k) of the tile's width, the
// 32-byte chunk m of row k at m ^ spread(k), where spread puts the eight rows that
// 32 lanes of a transposing read touch on all banks.
__device__ __forceinline__ int spread(int k) { return (k & 3) | ((k >> 1) & 4); }

struct Stage {
  ex_i32x4 buf;
  uint32_t mask, to;
};

// How a wave copies its part of an operand's stages: kN copies a stage.
template <int kRows, int kWaves, bool kAcross, bool kPairs>
struct StageCopy {
  static constexpr int kN = kRows / 8 / kWaves;
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
      constexpr int kRowBytes = kRows * 2, kPer = 1024 / kRowBytes;
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
  // Stage s, whose first k is k0 (of k); none of it is read if it is off.
  __device__ __forceinline__ Stage stage(int s, int k0, int k, bool on) const {
    const uint64_t at = (uint64_t)s * step;
    return {buffer_at(base + at, on ? left - (int64_t)at : 0),
            // along k: chunks past the last channel are zeros
            !kAcross && k0 + lane_k >= k ? kOutside : 0u, lds + (s & 1) * (kRows * 128)};
  }
  __device__ __forceinline__ void copy(const Stage &g, int i) const {
    copy16_bounded(g.buf, off[i] | g.mask, g.to + i * (kWaves * 1024));
  }
};

// Fragment t (16 rows from row t * 16), channels 32 kk ... + 31 of a stage.
template <int kRows, bool kAcross>
__device__ __forceinline__ bf16x8 fragment(const uint8_t *stage, int t, int kk) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
  if (kAcross) {
    constexpr int kRowBytes = kRows * 2;
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

// kRW x kCW waves, each with kRT x kCT fragments of 16.
template <int kRW, int kCW, int kRT, int kCT, bool kRAcross, bool kCAcross, int kAct>
__global__ __launch_bounds__(kRW *kCW * 64, kRW *kCW == 4 && kRT * kCT > 32 ? 1 : 2) void
product_kernel(ProductArgs a) {
  constexpr int kWaves = kRW * kCW, kR = kRW * kRT * 16, kC = kCW * kCT * 16;
  constexpr bool kPairs = kAct == kActSwiglu;
  __shared__ __align__(1024) uint8_t lds_r[2][kR * 128], lds_c[2][kC * 128];
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
  auto rows_of = [&](int s) { return cr.stage(s, k0 + s * kStep, a.k, s < n); };
  auto cols_of = [&](int s) { return cc.stage(s, k0 + s * kStep, a.k, s < n); };

  f32x4 acc[kRT][kCT];
#pragma unroll
  for (int i = 0; i < kRT; ++i)
#pragma unroll
    for (int j = 0; j < kCT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // A stage passes in 2 kRT slots of kCT products: first those of its channels 0-31,
  // whose fragments were read during the stage before, then those of 32-63, read
  // in the slots up to kRead. From slot kFree on, behind a barrier, the stage's LDS
  // is free, and the copies of the stage after next go there: they have more
  // than a stage's time to land. From slot kNext on, behind another barrier, the next
  // stage has landed and its first fragments are read. (Items of a read: the columns'
  // fragments 0 ... kCT - 1, then the rows'.)
  constexpr int kItems = kRT + kCT, kCopies = kRN + kCN, kSlots = 2 * kRT;
  constexpr int kRead = kRT * 5 / 8, kFree = kRT * 6 / 8, kNext = kRT * 3 / 2;
  constexpr int kReadPer = (kItems + kRead - 1) / kRead;
  constexpr int kNextPer = (kItems + kSlots - kNext - 1) / (kSlots - kNext);
  constexpr int kCopyPer = 2;
  static_assert((kSlots - kFree) * kCopyPer >= kCopies, "a stage's copies fit its slots");
  constexpr int kAhead = (kNext - kFree) * kCopyPer < kCopies ? (kNext - kFree) * kCopyPer : kCopies;
  bf16x8 fr[2][kRT], fc[2][kCT];
  auto read = [&](int s, int kk, int from, int to) {
    const uint8_t *sr = lds_r[s & 1], *sc = lds_c[s & 1];
#pragma unroll
    for (int m = from; m < to; ++m) {
      if (m < kCT)
        fc[kk][m] = fragment<kC, kCAcross>(sc, wc * kCT + m, kk);
      else if (m < kItems)
        fr[kk][m - kCT] = fragment<kR, kRAcross>(sr, wr * kRT + m - kCT, kk);
    }
  };
  auto copy = [&](const Stage &gr, const Stage &gc, int i) {
    if (i < kRN)
      cr.copy(gr, i);
    else if (i < kCopies)
      cc.copy(gc, i - kRN);
  };

#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const Stage gr = rows_of(s), gc = cols_of(s);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) copy(gr, gc, i);
  }
  __builtin_amdgcn_s_waitcnt(vmcnt(kCopies));
  lds_barrier();
  read(0, 0, 0, kItems);
  for (int s = 0; s < n; ++s) {
    const Stage gr = rows_of(s + 2), gc = cols_of(s + 2);
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      if (q < kRead) read(s, 1, q * kReadPer, (q + 1) * kReadPer);
      if (q == kFree) {
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      if (q == kNext) {
        __builtin_amdgcn_s_waitcnt(vmcnt(kAhead));
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      if (q >= kNext) read(s + 1, 0, (q - kNext) * kNextPer, (q - kNext + 1) * kNextPer);
      if (q >= kFree) {
#pragma unroll
        for (int c = 0; c < kCopyPer; ++c) copy(gr, gc, (q - kFree) * kCopyPer + c);
      }
      const int kk = q / kRT, i = q % kRT;
#pragma unroll
      for (int j = 0; j < kCT; ++j)
        acc[i][j] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(fc[kk][j], fr[kk][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __builtin_amdgcn_s_waitcnt(vmcnt(0));  // no copy outlives the workgroup

  const int l16 = lane & 15, quad = lane >> 4;
#pragma unroll
  for (int i = 0; i < kRT; ++i) {
    const int64_t t = row0 + (wr * kRT + i) * 16 + l16;
    if (t >= a.rows) continue;
    if (a.splits > 1) {  // as they are; a pair's halves in their own columns
#pragma unroll
      for (int j = 0; j < kCT; ++j) {
        int c = col0 + (wc * kCT + j) * 16 + quad * 4;
        int at = c;
        if (kPairs) {
          const int b = c >> 4;
          c = (b >> 1) * 16 + (c & 15);
          at = c + (b & 1) * a.e.N;
        }
        if (c < a.e.N)
          *reinterpret_cast<f32x4 *>(a.ws + ((int64_t)part * a.rows + t) *
                                                (kPairs ? 2 * (int64_t)a.e.N : a.e.N) + at) =
              acc[i][j];
      }
    } else if (kPairs) {
#pragma unroll
      for (int j = 0; j < kCT; j += 2) {
        const int c = (col0 + (wc * kCT + j) * 16) / 2 + quad * 4;
        if (c < a.e.N) linear_store<kAct>(a.e, t, c, acc[i][j], acc[i][j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kCT; ++j) {
        const int c = col0 + (wc * kCT + j) * 16 + quad * 4;
        if (c < a.e.N) linear_store<kAct>(a.e, t, c, acc[i][j], acc[i][j]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Adds the parts of a split product up, in order, and finishes them.
template <int kAct>
__global__ __launch_bounds__(256) void join_kernel(ProductArgs a) {
  const int NN = kAct == kActSwiglu ? 2 * a.e.N : a.e.N, quads = a.e.N / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.rows * quads) return;
  const int64_t t = i / quads;
  const int n = (int)(i - t * quads) * 4;
  const float *p = a.ws + t * NN + n;
  const int64_t part = (int64_t)a.rows * NN;
  f32x4 z = *reinterpret_cast<const f32x4 *>(p), up = z;
  if (kAct == kActSwiglu) up = *reinterpret_cast<const f32x4 *>(p + a.e.N);
  for (int s = 1; s < a.splits; ++s) {
    p += part;
    z += *reinterpret_cast<const f32x4 *>(p);
    if (kAct == kActSwiglu) up += *reinterpret_cast<const f32x4 *>(p + a.e.N);
  }
  linear_store<kAct>(a.e, t, n, z, up);
}

struct Plan {
  int tile;         // rows and columns of a tile: 256 or 128
  int splits, steps;  // parts of k and their stages
};

// Tiles of 256 x 256 where they fill the chip, else of 128 x 128; too few of
// those to fill it, k is split as far as that leaves a part eight stages.
Plan plan(int64_t rows, int64_t cols, int64_t k) {
  auto tiles = [&](int64_t t) { return ((rows + t - 1) / t) * ((cols + t - 1) / t); };
  const int64_t steps = (k + kStep - 1) / kStep;
  Plan p{256, 1, (int)steps};
  if (tiles(256) >= 192) return p;
  p.tile = 128;
  const int64_t n = tiles(128);
  int64_t s = 512 / n;
  if (s > steps / 8) s = steps / 8;
  const int64_t fit = kMaxWorkspace / 4 / (rows * cols);
  if (s > fit) s = fit;
  if (s > 1) {
    p.steps = (int)((steps + s - 1) / s);
    p.splits = (int)((steps + p.steps - 1) / p.steps);
  }
  return p;
}

template <bool kRAcross, bool kCAcross, int kAct>
hipError_t launch_product(ProductArgs a, hipStream_t s) {
  const int64_t cols = kAct == kActSwiglu ? 2 * (int64_t)a.e.N : a.e.N;
  a.cols = (int32_t)cols;
  const Plan p = plan(a.rows, cols, a.k);
  a.col_units = (int32_t)((cols + p.tile - 1) / p.tile);
  a.splits = p.splits;
  a.split_steps = p.steps;
  const int64_t units = (int64_t)a.col_units * ((a.rows + p.tile - 1) / p.tile) * p.splits;
  const dim3 grid((unsigned)((units + 7) / 8 * 8));
  if (p.tile == 256)
    hipLaunchKernelGGL((product_kernel<2, 2, 8, 8, kRAcross, kCAcross, kAct>), grid, dim3(256), 0,
                       s, a);
  else
    hipLaunchKernelGGL((product_kernel<2, 2, 4, 4, kRAcross, kCAcross, kAct>), grid, dim3(256), 0,
                       s, a);
  if (p.splits > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(join_kernel<kAct>,
                       dim3((unsigned)(((int64_t)a.rows * (a.e.N / 4) + 255) / 256)), dim3(256), 0,
                       s, a);
  }
  return hipGetLastError();
}

size_t plan_bytes(int64_t rows, int64_t cols, int64_t k) {
  if (rows == 0) return 0;
  const Plan p = plan(rows, cols, k);
  return p.splits > 1 ? (size_t)(p.splits * rows * cols * 4) : 0;
}

}  // namespace

size_t linear_workspace(int32_t T, int32_t N, int32_t C, int32_t act) {
  return plan_bytes(T, act == kActSwiglu ? 2 * (int64_t)N : N, C);
}
size_t linear_grad_workspace(int32_t T, int32_t N, int32_t C) {
  const size_t x = plan_bytes(T, C, N), w = plan_bytes(N, C, T);
  return x > w ? x : w;
}

hipError_t launch_linear(int32_t T, int32_t N, int32_t C, const uint16_t *x, const uint16_t *w,
                         const float *bias, const uint16_t *residual, void *out, uint16_t *pre,
                         int32_t act, bool f32, float *ws, hipStream_t s) {
  ProductArgs a{x, w, T, 0, C, C, C, 0, 1, 0, ws, {bias, residual, out, pre, N, f32}};
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
