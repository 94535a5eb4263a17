// Router with a balance bias and groups: among the experts of the best groups
// the K largest choices c = score + bias of each token, and their weights, from
// the scores alone.
//
// One wave holds one token, expert e = lane + 64 * j in register j. A choice is
// compared as a double: scores of different logits that a float would merge, or
// order wrongly by its rounding, still rank as they stand.
#include "gate.hpp"

namespace moe {
namespace {

constexpr uint64_t kNone = 0;  // the key of an expert that cannot be selected

__device__ __forceinline__ uint64_t choice_key(double c) {
  const int64_t u = (int64_t)__double_as_longlong(c + 0.0);
  return (uint64_t)u ^ ((uint64_t)(u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_choice(uint64_t k) {
  const int64_t u = (int64_t)k;
  return __longlong_as_double(u ^ (int64_t)((uint64_t)~(u >> 63) | 0x8000000000000000ull));
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t m) {
  for (int d = 32; d; d >>= 1) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)m, d);
    m = o > m ? o : m;
  }
  return m;
}
__device__ __forceinline__ double wave_sum_d(double x) {
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

struct GroupArgs {
  const void *x;
  const float *bias;  // nullptr: none
  int32_t T, E, K, G, KG;
  float scale;
  bool bf16, sum2;
  int64_t *idx;
  float *w;
  int32_t *status;
};

template <int V, int kMode>
__global__ __launch_bounds__(256) void gate_grouped_kernel(GroupArgs a) {
  constexpr bool kSig = kMode & kGateSigmoid;
  __shared__ uint64_t choices[4][V * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + wave));
  if (t >= a.T) return;
  const int E = a.E;
  bool bad = false;
  float x[V];
  gate_row<V>(a.x, (int64_t)t * E, E, a.bf16, x);
  uint64_t key[V];
  uint32_t top_key = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t k = gate_key(x[j], &bad);
    x[j] = lane + 64 * j < E && k ? key_logit(k) : -INFINITY;
    top_key = umax32(top_key, lane + 64 * j < E ? k : 0u);
  }
  top_key = wave_max_u(top_key);
  const float top = top_key ? key_logit(top_key) : 0.0f;
  double sum = 1.0;
  double p[V];
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = exp(kSig ? -(double)x[j] : (double)x[j] - (double)top);
  if (kSig) {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = 1.0 / (1.0 + p[j]);
  } else {
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) s += p[j];
    sum = wave_sum_d(s);
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] /= sum;
  }
  bool bad_bias = false;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    bool ok = x[j] != -INFINITY;
    double c = p[j];
    if (a.bias) {
      const float b = a.bias[min(lane + 64 * j, E - 1)];
      bool bb = false;
      if (gate_key(b, &bb) == 0) ok = false;
      bad_bias = bad_bias || bb;
      c += (double)b;
    }
    key[j] = ok ? choice_key(c) : kNone;
  }
  if (a.G > 1) {
    const int n = E / a.G;
#pragma unroll
    for (int j = 0; j < V; ++j) choices[wave][lane + 64 * j] = key[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    // lane g: group g
    uint64_t group = kNone;
    if (lane < a.G) {
      uint64_t k1 = kNone, k2 = kNone;
      for (int i = 0; i < n; ++i) {
        const uint64_t k = choices[wave][lane * n + i];
        const uint64_t lo = k < k1 ? k : k1;
        k1 = k > k1 ? k : k1;
        k2 = lo > k2 ? lo : k2;
      }
      group = k1;
      if (a.sum2 && k2 != kNone) group = choice_key(key_choice(k1) + key_choice(k2));
    }
    uint64_t kept = 0;
    for (int k = 0; k < a.KG; ++k) {
      const uint64_t m = wave_max_u64(group);
      if (m == kNone) break;
      const int g = __ffsll((unsigned long long)__ballot(group == m)) - 1;
      kept |= 1ull << g;
      if (lane == g) group = kNone;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (!(kept >> ((uint32_t)min(lane + 64 * j, E - 1) / (uint32_t)n) & 1)) key[j] = kNone;
  }
  int my_id = -1;
  float my_x = -INFINITY;
  for (int k = 0; k < a.K; ++k) {
    uint64_t head = key[0];
    int at = 0;
    float hx = x[0];
#pragma unroll
    for (int j = 1; j < V; ++j) {
      const bool up = key[j] > head;
      head = up ? key[j] : head;
      at = up ? j : at;
      hx = up ? x[j] : hx;
    }
    const uint64_t m = wave_max_u64(head);
    if (m == kNone) break;
    uint64_t tied = __ballot(head == m);
    int l = __ffsll((unsigned long long)tied) - 1;
    int id = l + 64 * __builtin_amdgcn_readlane(at, l);
    while (tied &= tied - 1) {  // uniform
      const int l2 = __ffsll((unsigned long long)tied) - 1;
      const int id2 = l2 + 64 * __builtin_amdgcn_readlane(at, l2);
      if (id2 < id) {
        id = id2;
        l = l2;
      }
    }
    const float bx = lane_f(hx, l);
    if (lane == k) {
      my_id = id;
      my_x = bx;
    }
    if (lane == l) {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = j == at ? kNone : key[j];
    }
  }
  const float s = gate_score<kMode>(my_x, top, (float)sum);
  if (lane < a.K) {
    const int64_t o = (int64_t)t * a.K + lane;
    a.idx[o] = my_id;
    a.w[o] = my_id < 0 ? 0.0f : s * a.scale;
  }
  if (a.status && __ballot(bad || bad_bias) && lane == 0) atomicOr(a.status, kStBadLogit);
}

template <int V, int kMode>
hipError_t gate_grouped_vm(const GroupArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((gate_grouped_kernel<V, kMode>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0,
                     s, a);
  return hipGetLastError();
}
template <int kMode>
hipError_t gate_grouped_m(const GroupArgs &a, hipStream_t s) {
  if (a.E <= 64) return gate_grouped_vm<1, kMode>(a, s);
  if (a.E <= 128) return gate_grouped_vm<2, kMode>(a, s);
  if (a.E <= 256) return gate_grouped_vm<4, kMode>(a, s);
  if (a.E <= 512) return gate_grouped_vm<8, kMode>(a, s);
  return gate_grouped_vm<16, kMode>(a, s);
}

}  // namespace

hipError_t launch_gate_grouped(const void *x, const float *bias, int32_t T, int32_t E, int32_t K,
                               int32_t G, int32_t KG, int32_t flags, float scale, int64_t *idx,
                               float *w, int32_t *status, hipStream_t s) {
  const GroupArgs a{x,   bias, T, E, K, G, KG, scale, (flags & kGateBf16) != 0,
                    (flags & kGateGroupSum2) != 0, idx, w, status};
  switch (flags & (kGateSigmoid | kGateRenorm)) {
    case 0: return gate_grouped_m<0>(a, s);
    case kGateSigmoid: return gate_grouped_m<kGateSigmoid>(a, s);
    case kGateRenorm: return gate_grouped_m<kGateRenorm>(a, s);
    default: return gate_grouped_m<kGateSigmoid | kGateRenorm>(a, s);
  }
}

}  // namespace moe
