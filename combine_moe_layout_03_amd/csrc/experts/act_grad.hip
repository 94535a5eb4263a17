// Gradient of the dense product's epilogue:
//   d_z = act'(z) d_out   (SwiGLU: both halves),   d_bias = sum over the rows of d_z.
//
// A stream over the rows: a wave takes 512 columns of d_out (8 a lane) and every
// fourth row of its workgroup's run, adds its columns up in registers, and the
// workgroup writes one row of partial sums, which a second kernel adds in order.
// The sums are of the float d_z, before its rounding to bf16.
//
// Bound by bytes, nearly: 8192 rows of 2 x 2048 (SwiGLU) 176 MB in 33 us, 5.3 TB/s; two
// thirds of the vector unit's time is in use beside it. GELU, 1001 rows of 2824: 7 us
// (14 with the library's erfc and exp), a launch and few rows for each wave; their sums
// 2.6 us. Twice as many workgroups with half the rows: the same, and twice the partial
// sums.
#include "linear.hpp"

namespace moe {
namespace {

struct ActGradArgs {
  const ex_u32x4 *d_out, *z;
  ex_u32x4 *d_z;   // nullptr without an activation
  float *partial;  // [runs][columns of z], nullptr: no d_bias
  int32_t T, nv;   // rows, vectors of a row of d_out
  int32_t run;     // rows of a workgroup
};

template <int kAct>
__device__ __forceinline__ float slope(float z) {
  if (kAct == kActGelu) {
    const Normal n = normal(z);
    return __builtin_fmaf(z, n.density, n.below);
  }
  const Sigmoids g = sigmoids(z);
  return g.s * __builtin_fmaf(z, g.rest, 1.0f);
}

template <int kAct>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a) {
  constexpr bool kPairs = kAct == kActSwiglu;
  constexpr int kHalves = kPairs ? 2 : 1;
  __shared__ float join[4][kHalves][512];
  const int lane = threadIdx.x & 63, wave = scalar_i(threadIdx.x >> 6);
  const int v = blockIdx.x * 64 + lane, at = min(v, a.nv - 1);
  const bool ok = v < a.nv;
  float sum[kHalves][8];
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
#pragma unroll
    for (int d = 0; d < 8; ++d) sum[h][d] = 0.0f;
  const int end = min(a.T, ((int)blockIdx.y + 1) * a.run);
  struct Row {
    ex_u32x4 e, z, u;
  };
  auto load = [&](int t) {
    Row r;
    const int64_t row = (int64_t)t * a.nv * kHalves + at;
    r.e = __builtin_nontemporal_load(a.d_out + (int64_t)t * a.nv + at);
    r.z = kAct != kActNone ? __builtin_nontemporal_load(a.z + row) : r.e;
    r.u = kPairs ? __builtin_nontemporal_load(a.z + row + a.nv) : r.e;
    return r;
  };
  int t = blockIdx.y * a.run + wave;
  Row next = load(min(t, end - 1));
  for (; t < end; t += 4) {
    const ex_u32x4 e = next.e, z = next.z, u = next.u;
    ex_u32x4 dz, du;
    next = load(min(t + 4, end - 1));
    const int64_t row = (int64_t)t * a.nv * kHalves + at;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float g[2], k[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float d = b ? ex_hi(e[j]) : ex_lo(e[j]), x = b ? ex_hi(z[j]) : ex_lo(z[j]);
        g[b] = d;
        k[b] = 0.0f;
        if (kPairs) {
          const float w = b ? ex_hi(u[j]) : ex_lo(u[j]);
          g[b] = d * slope<kActSilu>(x) * w;
          k[b] = d * activation<kActSilu>(x);
          sum[kHalves - 1][2 * j + b] += k[b];
        } else if (kAct != kActNone) {
          g[b] = d * slope<kAct>(x);
        }
        sum[0][2 * j + b] += g[b];
      }
      dz[j] = ex_round2(g[0], g[1]);
      du[j] = ex_round2(k[0], k[1]);
    }
    if (kAct != kActNone && ok) {
      __builtin_nontemporal_store(dz, a.d_z + row);
      if (kPairs) __builtin_nontemporal_store(du, a.d_z + row + a.nv);
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
#pragma unroll
    for (int d = 0; d < 8; ++d) join[wave][h][lane * 8 + d] = sum[h][d];
  lds_barrier();
  float *to = a.partial + (int64_t)blockIdx.y * a.nv * 8 * kHalves + (int64_t)blockIdx.x * 512;
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
    for (int i = threadIdx.x; i < 512; i += 256)
      if ((int)blockIdx.x * 512 + i < a.nv * 8)
        to[(int64_t)h * a.nv * 8 + i] =
            (join[0][h][i] + join[1][h][i]) + (join[2][h][i] + join[3][h][i]);
}

// Runs of rows: about four workgroups a CU, and partial sums within kMaxWorkspace.
int32_t run_rows(int32_t T, int32_t nv, int32_t halves) {
  const int64_t blocks = (nv + 63) / 64;
  int64_t runs = 1024 / blocks;
  const int64_t fit = kMaxWorkspace / 4 / ((int64_t)nv * 8 * halves);
  if (runs > fit) runs = fit;
  if (runs < 1) runs = 1;
  int64_t rows = (T + runs - 1) / runs;
  return (int32_t)(rows < 8 ? 8 : (rows + 3) / 4 * 4);
}

}  // namespace

size_t act_grad_workspace(int32_t T, int32_t N, int32_t act) {
  if (T == 0) return 0;
  const int32_t halves = act == kActSwiglu ? 2 : 1, run = run_rows(T, N / 8, halves);
  return (size_t)((T + run - 1) / run) * N * halves * 4;
}

hipError_t launch_act_grad(int32_t T, int32_t N, const uint16_t *d_out, const uint16_t *z,
                           uint16_t *d_z, float *d_bias, int32_t act, float *ws, hipStream_t s) {
  const int32_t halves = act == kActSwiglu ? 2 : 1, nv = N / 8, run = run_rows(T, nv, halves);
  const int32_t runs = (T + run - 1) / run;
  const ActGradArgs a{reinterpret_cast<const ex_u32x4 *>(d_out),
                      reinterpret_cast<const ex_u32x4 *>(z),
                      reinterpret_cast<ex_u32x4 *>(d_z),
                      !d_bias ? nullptr : runs == 1 ? d_bias : ws,
                      T,
                      nv,
                      run};
  const dim3 grid((nv + 63) / 64, runs), block(256);
  switch (act) {
    case kActNone: hipLaunchKernelGGL(act_grad_kernel<kActNone>, grid, block, 0, s, a); break;
    case kActSilu: hipLaunchKernelGGL(act_grad_kernel<kActSilu>, grid, block, 0, s, a); break;
    case kActGelu: hipLaunchKernelGGL(act_grad_kernel<kActGelu>, grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL(act_grad_kernel<kActSwiglu>, grid, block, 0, s, a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !d_bias || runs == 1) return e;  // one run's sums are the result
  return launch_column_sum(ws, runs, N * halves, d_bias, s);
}

}  // namespace moe
