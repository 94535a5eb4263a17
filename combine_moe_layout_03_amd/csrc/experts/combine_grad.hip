// Gradient of the weighted combine out[t] = sum_k w[t,k] * y[slot[t,k]]:
//   dy[slot[t,k]] = w[t,k] * dout[t],   dw[t,k] = <dout[t], y[slot[t,k]]>.
//
// One workgroup of four waves per (token, k) pair: it reads the token's row of
// dout and the pair's row of y once, writes the pair's row of dy, and adds the
// products up in registers, over the wave and over the four waves in a fixed
// order: no atomics, so a repeated call gives the same bits. The K workgroups
// of a token are numbered 8 apart, which puts them on one XCD, where the
// token's row comes from L2 after the first of them (counted at 8192 x 8 x 7168:
// 1062 MB read from memory, 1057 MB of y and d_out).
//
// Bound by the bytes of y and d_y, rows at random places both ways. 8192 x 8 x
// 7168: 362 us (2.0 GB, 5.5 TB/s; a large copy reaches 6.1; 128 or 512 threads, or
// the loads of d_out ahead of the slot's check, change it by 1%, loads or stores
// not marked nontemporal cost 5 to 8%); 4096 x 6 x 4096 with a masked rank, whose
// rows of y are not read: 70 us (378 MB, 5.4 TB/s); 128 x 8 x 7168: 8 us, launch
// and one row's latency.
#include "experts.hpp"

namespace moe {
namespace {

constexpr int kCgThreads = 256;
constexpr int kCgVec = 4;  // 16-byte vectors in flight per lane and array

template <bool kDw>
__global__ __launch_bounds__(kCgThreads) void combine_grad_kernel(
    const int32_t *__restrict__ slot, const ex_u32x4 *__restrict__ dout,
    const ex_u32x4 *__restrict__ y, const float *__restrict__ w, int64_t rows, int32_t T,
    int32_t K, int32_t nvec, ex_u32x4 *__restrict__ dy, float *__restrict__ dw, CombineMask cm,
    int32_t *status) {
  __shared__ float part[kCgThreads / 64];
  // pair of this workgroup: tokens in groups of 8, the group's token fastest
  const uint32_t b = blockIdx.x, grp = b / (8u * K);
  const int r = (int)(b - grp * 8u * K);
  const int64_t t = (int64_t)grp * 8 + (r & 7);
  const int k = r >> 3;
  if (t >= T) return;
  const int64_t pair = t * K + k;
  const int32_t s = slot[pair];
  const bool ok = s >= 0 && s < rows;
  if (!ok) {
    if (threadIdx.x == 0) {
      if (kDw) dw[pair] = 0.0f;
      if (s != -1 && status) atomicOr(status, kStBadSlot);
    }
    return;
  }
  bool off = false;
  if (cm.idx) {
    const int64_t e = cm.idx[pair];
    off = e >= 0 && e < cm.E && cm.mask[rank_of((int)e, cm.l_magic)] != 0;
  }
  const float a = w ? w[pair] : 1.0f;
  const ex_u32x4 *src = dout + t * nvec;
  const ex_u32x4 *yr = y + (int64_t)s * nvec;
  ex_u32x4 *dst = dy + (int64_t)s * nvec;
  if (off) {
    for (int v = threadIdx.x; v < nvec; v += kCgThreads)
      __builtin_nontemporal_store(ex_u32x4(0u), dst + v);
    if (kDw && threadIdx.x == 0) dw[pair] = 0.0f;
    return;
  }
  float acc = 0.0f;
  for (int v0 = threadIdx.x; v0 < nvec; v0 += kCgThreads * kCgVec) {
    ex_u32x4 g[kCgVec], q[kCgVec];
#pragma unroll
    for (int i = 0; i < kCgVec; ++i) {
      const int v = min(v0 + i * kCgThreads, nvec - 1);
      g[i] = src[v];
      if (kDw) q[i] = __builtin_nontemporal_load(yr + v);
    }
#pragma unroll
    for (int i = 0; i < kCgVec; ++i) {
      const int v = v0 + i * kCgThreads;
      if (v >= nvec) continue;
      ex_u32x4 o;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float lo = ex_lo(g[i][c]), hi = ex_hi(g[i][c]);
        // the product is rounded to float, then to bf16: the first rounding is
        // 2^-16 of the second
        o[c] = ex_bf16x2(a * lo, a * hi);
        if (kDw) {
          acc = __builtin_fmaf(lo, ex_lo(q[i][c]), acc);
          acc = __builtin_fmaf(hi, ex_hi(q[i][c]), acc);
        }
      }
      __builtin_nontemporal_store(o, dst + v);
    }
  }
  if (kDw) {
    const float s0 = wave_sum_f(acc);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s0;
    __syncthreads();
    if (threadIdx.x == 0) dw[pair] = (part[0] + part[1]) + (part[2] + part[3]);
  }
}

}  // namespace

hipError_t launch_combine_grad(const uint16_t *dout, const uint16_t *y, int64_t rows,
                               const int32_t *slot, const float *w, uint16_t *dy, float *dw,
                               int32_t T, int32_t K, int32_t H, const CombineMask &mask,
                               int32_t *status, hipStream_t s) {
  if (T <= 0) return hipSuccess;
  const int64_t wgs = ((int64_t)T + 7) / 8 * 8 * K;
  const auto *d4 = reinterpret_cast<const ex_u32x4 *>(dout);
  const auto *y4 = reinterpret_cast<const ex_u32x4 *>(y);
  auto *o4 = reinterpret_cast<ex_u32x4 *>(dy);
  if (dw)
    hipLaunchKernelGGL((combine_grad_kernel<true>), dim3((unsigned)wgs), dim3(kCgThreads), 0, s,
                       slot, d4, y4, w, rows, T, K, H / 8, o4, dw, mask, status);
  else
    hipLaunchKernelGGL((combine_grad_kernel<false>), dim3((unsigned)wgs), dim3(kCgThreads), 0, s,
                       slot, d4, y4, w, rows, T, K, H / 8, o4, dw, mask, status);
  return hipGetLastError();
}

}  // namespace moe
