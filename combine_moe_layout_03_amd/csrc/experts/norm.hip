// Root-mean-square norm of the residual stream, and its gradient.
//
//   sum = bf16(x + residual),  rstd = 1 / sqrt(mean(sum^2) + eps),  n = sum * rstd
//   y = n * weight, written in bf16 and / or cast to E4M3 (as the FP8 dispatch casts)
// and back, with g = d_y * weight,
//   d_x = d_sum + rstd * (g - n * mean(g * n)),  d_weight = sum over the rows of d_y * n.
//
// A row stays in the registers of the threads that read it (8 channels a
// thread and vector), so every tensor passes once, but for the widest gradients'. The
// mean is float: 8 squares a lane and vector in order, then the lanes, then the waves,
// always alike. y is rounded once, from the sum as it is stored, so that the gradient, which has only
// that, sees the same n. The codes are those of the float y.
// d_weight: a workgroup adds its rows up in registers and writes one row of
// partial sums; a second kernel adds those in order.
//
// Bound by bytes. 8192 rows of 7168: 470 MB in 71 us (6.6 TB/s; a large copy reaches
// 6.1), the gradient as many and 15 MB of partial sums in 81 us (5.8), their sum 4 us;
// 4096 rows of 4096 with codes: 152 MB in 26 us, the gradient 25.7. The gradient was
// bound by instructions (97 us) while it rounded in integer arithmetic, the conversion
// instruction does two values at once, and unpacked the weight from memory for every
// row. A row is loaded while the one before it is computed: two workgroups of a CU
// then keep 96 KB in flight. 16 rows of 7168 with codes: 3.9 us, most of it the launch
// and two trips to memory; a row over 16 waves instead of 4 took 1.1 us off.
// Between 8192 and 16384 channels the gradient fills a SIMD's registers with one wave:
// 4096 x 12288 in 88 us, 4.6 TB/s (the norm 63, 6.4). Above, a row's values and sums
// pass the 128 registers of each of 1024 threads: the row is read twice, the second time
// from cache, one vector of a thread at a time. 2048 x 18432 in 75 us with the weight's
// sums, 4.0 TB/s; kept, the values lay in scratch memory (1464 us, and 1480 bytes a lane
// that the runtime had to allocate).
#include "cast.hpp"

namespace moe {
namespace {

__device__ __forceinline__ void unpack(ex_u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = ex_lo(v[j]);
    f[2 * j + 1] = ex_hi(v[j]);
  }
}
__device__ __forceinline__ ex_u32x4 pack(const float (&f)[8]) {
  return ex_u32x4{ex_round2(f[0], f[1]), ex_round2(f[2], f[3]), ex_round2(f[4], f[5]),
                  ex_round2(f[6], f[7])};
}

// Sum over the kWaves waves that share a row (one: over the wave). `part` is
// LDS of kWaves floats that the previous call did not use.
template <int kWaves>
__device__ __forceinline__ float row_sum(float x, float *part) {
  x = wave_sum_f(x);
  if (kWaves == 1) return x;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  lds_barrier();
  float s = part[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += part[w];
  return s;
}

struct NormArgs {
  const ex_u32x4 *x, *res;  // res nullptr: no residual
  const ex_u32x4 *weight;
  ex_u32x4 *sum, *y;  // nullptr: not written
  ex_u32x2 *q;
  float *fscale;
  uint32_t *wscale;
  int32_t T, nv;  // rows, 16-byte vectors of a row
  float h, eps;  // the row's length
};

// V vectors per thread; a workgroup takes one row (kWaves waves) or four (one
// wave each).
template <int kWaves, int V, bool kFp8, int kFlags>
__global__ __launch_bounds__(kWaves == 1 ? 256 : kWaves * 64) void norm_kernel(NormArgs a) {
  constexpr int kStride = kWaves * 64;
  __shared__ float part[kWaves];
  const int tid = kWaves == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int row = __builtin_amdgcn_readfirstlane(
      kWaves == 1 ? (int)(blockIdx.x * 4 + (threadIdx.x >> 6)) : (int)blockIdx.x);
  if (row >= a.T) return;
  const int64_t at = (int64_t)row * a.nv;
  ex_u32x4 v[V], w[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = min(tid + j * kStride, a.nv - 1);
    v[j] = __builtin_nontemporal_load(a.x + at + i);
    w[j] = a.weight[i];
  }
  if (a.res) {
    ex_u32x4 r[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      r[j] = __builtin_nontemporal_load(a.res + at + min(tid + j * kStride, a.nv - 1));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float f[8], g[8];
      unpack(v[j], f);
      unpack(r[j], g);
#pragma unroll
      for (int d = 0; d < 8; ++d) f[d] += g[d];
      v[j] = pack(f);
      if (a.sum && tid + j * kStride < a.nv) a.sum[at + tid + j * kStride] = v[j];
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float f[8];
    unpack(v[j], f);
    float s = 0.0f;
#pragma unroll
    for (int d = 0; d < 8; ++d) s = __builtin_fmaf(f[d], f[d], s);
    ss += tid + j * kStride < a.nv ? s : 0.0f;
  }
  const float mean = row_sum<kWaves>(ss, part) / a.h;
  const float rstd = 1.0f / sqrtf(mean + a.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * kStride;
    const bool ok = i < a.nv;
    float f[8], g[8];
    unpack(v[j], f);
    unpack(w[j], g);
#pragma unroll
    for (int d = 0; d < 8; ++d) f[d] = f[d] * rstd * g[d];
    if (a.y && ok) __builtin_nontemporal_store(pack(f), a.y + at + i);
    if (kFp8) {
      // (whole 16-lane groups are inside or outside of the row)
      const uint32_t top = row16_max(largest(f));
      const float s = group_scale<kFlags>(top, top >= kInfBits);
      if (ok) __builtin_nontemporal_store(group_codes(f, s), a.q + at + i);
      if (kFlags & kFp8Ue8m0) {  // whole waves are
        const uint32_t word = ue8m0_word(s);
        if (ok && (tid & 63) == 0) a.wscale[(int64_t)row * (a.nv >> 6) + (i >> 6)] = word;
      } else if (ok && (tid & 15) == 0) {
        a.fscale[(int64_t)row * (a.nv >> 4) + (i >> 4)] = s;
      }
    }
  }
}

struct NormGradArgs {
  const ex_u32x4 *sum, *weight, *dy, *dsum;  // dsum nullptr: 0
  ex_u32x4 *dx;
  float *partial;  // [gridDim.x][H], nullptr: no d_weight
  int32_t T, nv;
  float h, eps;  // the row's length
};

// A workgroup takes rows blockIdx.x, + gridDim.x, ...; with one wave a row, four
// at a time, whose sums for the weight are joined at the end.
template <int kWaves, int V>
__global__ __launch_bounds__(kWaves == 1 ? 256 : kWaves * 64) void norm_grad_kernel(
    NormGradArgs a) {
  constexpr int kStride = kWaves * 64, kRows = kWaves == 1 ? 4 : 1;
  __shared__ float part[2][2 * kWaves];
  __shared__ float join[kWaves == 1 ? 4 * 64 * 8 : 1];
  const int tid = kWaves == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float dw[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int d = 0; d < 8; ++d) dw[j][d] = 0.0f;
  int turn = 0;
  // The widest rows do not fit the registers beside their sums for the weight: each
  // vector is loaded where it is used, for the row's sums and again for its gradient.
  constexpr bool kHeld = kWaves * V <= 64;
  constexpr int kHold = kHeld ? V : 1;
  struct Row {
    ex_u32x4 v[kHold], e[kHold], ds[kHold];
  };
  auto load = [&](int row) {
    Row r;
    const int64_t at = (int64_t)row * a.nv;
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int i = min(tid + j * kStride, a.nv - 1);
      r.v[j] = __builtin_nontemporal_load(a.sum + at + i);
      r.e[j] = __builtin_nontemporal_load(a.dy + at + i);
      r.ds[j] = a.dsum ? __builtin_nontemporal_load(a.dsum + at + i) : ex_u32x4{0, 0, 0, 0};
    }
    return r;
  };
  ex_u32x4 weight[kHold];
#pragma unroll
  for (int j = 0; j < kHold; ++j) weight[j] = a.weight[min(tid + j * kStride, a.nv - 1)];
  const int step = (int)gridDim.x * kRows;
  int row = (int)blockIdx.x * kRows + (kWaves == 1 ? wave : 0);
  if (row >= a.T && kWaves > 1) return;  // (no workgroup is without a row)
  Row next;
  if (kHeld) next = load(min(row, a.T - 1));
  for (; row < a.T; row += step, turn ^= 1) {
    Row now;
    if (kHeld) {
      now = next;
      next = load(min(row + step, a.T - 1));  // the last one's again behind the end
    }
    const int64_t at = (int64_t)row * a.nv;
    float ss = 0.0f, gs = 0.0f;  // of squares, and of sum * g (rstd follows)
    int self = tid;  // (new to the compiler each time, which would keep values and addresses)
    if (!kHeld) asm volatile("" : "+v"(self));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (!kHeld && j * kStride >= a.nv) continue;  // uniform
      const int k = min(self + j * kStride, a.nv - 1);
      float f[8], g[8], w[8];
      unpack(kHeld ? now.v[j % kHold] : a.sum[at + k], f);
      unpack(kHeld ? now.e[j % kHold] : a.dy[at + k], g);
      unpack(kHeld ? weight[j % kHold] : a.weight[k], w);
      float s = 0.0f, t = 0.0f;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        s = __builtin_fmaf(f[d], f[d], s);
        t = __builtin_fmaf(f[d], g[d] * w[d], t);
      }
      const bool ok = tid + j * kStride < a.nv;
      ss += ok ? s : 0.0f;
      gs += ok ? t : 0.0f;
    }
    ss = wave_sum_f(ss);
    gs = wave_sum_f(gs);
    if (kWaves > 1) {
      float *p = part[turn];
      if ((threadIdx.x & 63) == 0) {
        p[wave] = ss;
        p[kWaves + wave] = gs;
      }
      lds_barrier();
      ss = p[0];
      gs = p[kWaves];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        ss += p[w];
        gs += p[kWaves + w];
      }
    }
    const float rstd = 1.0f / sqrtf(ss / a.h + a.eps);
    const float c = gs * rstd / a.h;  // mean(g n)
    if (!kHeld) asm volatile("" : "+v"(self)::"memory");
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (!kHeld && j * kStride >= a.nv) continue;
      const int i = self + j * kStride, k = min(i, a.nv - 1);
      float f[8], g[8], w[8], o[8];
      unpack(kHeld ? now.v[j % kHold] : __builtin_nontemporal_load(a.sum + at + k), f);
      unpack(kHeld ? now.e[j % kHold] : __builtin_nontemporal_load(a.dy + at + k), g);
      unpack(kHeld ? weight[j % kHold] : a.weight[k], w);
      if (kHeld)
        unpack(now.ds[j % kHold], o);
      else
        unpack(a.dsum ? __builtin_nontemporal_load(a.dsum + at + k) : ex_u32x4{0, 0, 0, 0}, o);
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const float n = f[d] * rstd;
        dw[j][d] = __builtin_fmaf(g[d], n, dw[j][d]);
        o[d] = __builtin_fmaf(rstd, __builtin_fmaf(-n, c, g[d] * w[d]), o[d]);
      }
      if (i < a.nv) __builtin_nontemporal_store(pack(o), a.dx + at + i);
    }
  }
  if (!a.partial) return;
  float *to = a.partial + (int64_t)blockIdx.x * a.nv * 8;
  if (kWaves == 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      lds_barrier();
#pragma unroll
      for (int d = 0; d < 8; ++d) join[(wave * 64 + tid) * 8 + d] = dw[j][d];
      lds_barrier();
      for (int k = threadIdx.x; k < 512; k += 256) {
        const float s = (join[k] + join[512 + k]) + (join[1024 + k] + join[1536 + k]);
        if (j * 64 + (k >> 3) < a.nv) to[j * 512 + k] = s;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * kStride;
    if (i >= a.nv) continue;
    float4 *o = reinterpret_cast<float4 *>(to + (int64_t)i * 8);
    o[0] = float4{dw[j][0], dw[j][1], dw[j][2], dw[j][3]};
    o[1] = float4{dw[j][4], dw[j][5], dw[j][6], dw[j][7]};
  }
}

// out[i] = sum over the P rows of partial[p][i], in an order that depends on P
// alone. A workgroup takes 32 columns, a line of every row; its 32 half waves
// share the rows out, eight loads of each in flight.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float *__restrict__ partial,
                                                          int32_t P, int32_t n,
                                                          float *__restrict__ out) {
  __shared__ float part[32][33];
  const int col = threadIdx.x & 31, group = threadIdx.x >> 5;
  const float *p = partial + min((int)blockIdx.x * 32 + col, n - 1);
  float s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = 0.0f;
  for (int r = group; r < P; r += 256) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = p[(int64_t)min(r + 32 * k, P - 1) * n];
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] += r + 32 * k < P ? v[k] : 0.0f;
  }
  part[group][col] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  lds_barrier();
  if (threadIdx.x >= 32) return;
  float t = 0.0f;
#pragma unroll
  for (int g = 0; g < 32; ++g) t += part[g][col];
  if ((int)blockIdx.x * 32 + col < n) out[blockIdx.x * 32 + col] = t;
}

__global__ __launch_bounds__(256) void zeros_kernel(float *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0.0f;
}

// How a row is spread: one wave where a wave's registers hold it and there are
// rows for all CUs, else a workgroup.
struct Spread {
  int waves, v;  // waves of a row, vectors of a thread
};
Spread spread(int32_t T, int32_t nv) {
  if (nv <= 64) return {1, 1};
  if (nv <= 128 && T >= 512) return {1, 2};
  if (nv <= 256 && T >= 512) return {1, 4};
  if (nv <= 256) return {4, 1};
  if (nv <= 1024 && T <= 256) return {16, 1};
  if (nv <= 512) return {4, 2};
  if (nv <= 1024) return {4, 4};
  if (nv <= 2048) return {4, 8};
  return {16, 8};
}

template <int kWaves, int V>
hipError_t norm_wv(const NormArgs &a, bool fp8, int32_t flags, hipStream_t s) {
  const dim3 grid(kWaves == 1 ? (a.T + 3) / 4 : a.T), block(kWaves == 1 ? 256 : kWaves * 64);
  if (!fp8)
    hipLaunchKernelGGL((norm_kernel<kWaves, V, false, 0>), grid, block, 0, s, a);
  else if (flags & kFp8Ue8m0)
    hipLaunchKernelGGL((norm_kernel<kWaves, V, true, kFp8RoundScale | kFp8Ue8m0>), grid, block, 0,
                       s, a);
  else if (flags & kFp8RoundScale)
    hipLaunchKernelGGL((norm_kernel<kWaves, V, true, kFp8RoundScale>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((norm_kernel<kWaves, V, true, 0>), grid, block, 0, s, a);
  return hipGetLastError();
}
template <int kWaves, int V>
hipError_t norm_grad_wv(const NormGradArgs &a, int32_t blocks, hipStream_t s) {
  hipLaunchKernelGGL((norm_grad_kernel<kWaves, V>), dim3(blocks),
                     dim3(kWaves == 1 ? 256 : kWaves * 64), 0, s, a);
  return hipGetLastError();
}

#define MOE_BY_SPREAD(FN, SP, ...)                                   \
  do {                                                               \
    if (SP.waves == 1 && SP.v == 1) return FN<1, 1>(__VA_ARGS__);    \
    if (SP.waves == 1 && SP.v == 2) return FN<1, 2>(__VA_ARGS__);    \
    if (SP.waves == 1) return FN<1, 4>(__VA_ARGS__);                 \
    if (SP.waves == 16 && SP.v == 1) return FN<16, 1>(__VA_ARGS__);  \
    if (SP.waves == 16) return FN<16, 8>(__VA_ARGS__);               \
    if (SP.v == 1) return FN<4, 1>(__VA_ARGS__);                     \
    if (SP.v == 2) return FN<4, 2>(__VA_ARGS__);                     \
    if (SP.v == 4) return FN<4, 4>(__VA_ARGS__);                     \
    return FN<4, 8>(__VA_ARGS__);                                    \
  } while (0)

hipError_t norm_grad_launch(const NormGradArgs &a, const Spread &sp, int32_t blocks,
                            hipStream_t s) {
  MOE_BY_SPREAD(norm_grad_wv, sp, a, blocks, s);
}

}  // namespace

hipError_t launch_column_sum(const float *partial, int32_t P, int32_t n, float *out,
                             hipStream_t s) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((n + 31) / 32), dim3(1024), 0, s, partial, P, n, out);
  return hipGetLastError();
}

hipError_t launch_zeros(float *p, int64_t n, hipStream_t s) {
  const int64_t blocks = (n + 255) / 256;
  hipLaunchKernelGGL(zeros_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s,
                     p, n);
  return hipGetLastError();
}

hipError_t launch_rms_norm(int32_t T, int32_t H, const uint16_t *x, const uint16_t *residual,
                           const uint16_t *weight, float eps, uint16_t *sum, uint16_t *y,
                           uint8_t *q, void *scale, int32_t flags, hipStream_t s) {
  const NormArgs a{reinterpret_cast<const ex_u32x4 *>(x),
                   reinterpret_cast<const ex_u32x4 *>(residual),
                   reinterpret_cast<const ex_u32x4 *>(weight),
                   reinterpret_cast<ex_u32x4 *>(sum),
                   reinterpret_cast<ex_u32x4 *>(y),
                   reinterpret_cast<ex_u32x2 *>(q),
                   static_cast<float *>(scale),
                   static_cast<uint32_t *>(scale),
                   T,
                   H / 8,
                   (float)H,
                   eps};
  const Spread sp = spread(T, a.nv);
  MOE_BY_SPREAD(norm_wv, sp, a, q != nullptr, flags, s);
}

// Workgroups of the gradient, and so rows of partial sums: two for every CU, as
// far as there are rows and the partial sums stay within kMaxWorkspace. Up to four
// rows (of workgroups) are one workgroup's, whose sums are the weight's gradient
// itself: 2 us more for it, a second launch less.
int32_t norm_grad_blocks(int32_t T, int32_t H) {
  const Spread sp = spread(T, H / 8);
  const int64_t rows = sp.waves == 1 ? ((int64_t)T + 3) / 4 : T;
  int64_t n = sp.waves == 16 && sp.v > 1 ? 256 : 512;
  if (n > rows) n = rows;
  if (rows <= 4) n = 1;
  if (n > kMaxWorkspace / 4 / H) n = kMaxWorkspace / 4 / H;
  return (int32_t)n;
}

hipError_t launch_rms_norm_grad(int32_t T, int32_t H, const uint16_t *sum, const uint16_t *weight,
                                float eps, const uint16_t *d_y, const uint16_t *d_sum,
                                uint16_t *d_x, float *d_weight, float *ws, hipStream_t s) {
  const int32_t blocks = norm_grad_blocks(T, H);
  // (the kernel stores its sums in vectors)
  const bool direct = blocks == 1 && (reinterpret_cast<uintptr_t>(d_weight) & 15u) == 0;
  const NormGradArgs a{reinterpret_cast<const ex_u32x4 *>(sum),
                       reinterpret_cast<const ex_u32x4 *>(weight),
                       reinterpret_cast<const ex_u32x4 *>(d_y),
                       reinterpret_cast<const ex_u32x4 *>(d_sum),
                       reinterpret_cast<ex_u32x4 *>(d_x),
                       !d_weight ? nullptr : direct ? d_weight : ws,
                       T,
                       H / 8,
                       (float)H,
                       eps};
  const hipError_t e = norm_grad_launch(a, spread(T, a.nv), blocks, s);
  if (e != hipSuccess || !d_weight || direct) return e;
  return launch_column_sum(ws, blocks, H, d_weight, s);
}
#undef MOE_BY_SPREAD

}  // namespace moe
