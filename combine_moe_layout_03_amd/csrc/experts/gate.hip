// Router: top-k experts of each token and their weights, and the gradient of
// the weights with respect to the logits.
//
// One wave holds one token's E <= 1024 logits, expert e = lane + 64 * j in
// register j, as unsigned keys whose integer order is the float order (the sign
// bit flipped, negatives complemented), 0 for an expert that cannot be
// selected. A lane sorts its keys once (for up to four of them); then K times:
// the largest head of the 64 lanes (six DPP steps), the lane that holds it (a
// ballot), whose list moves up. Several lanes with the same key, rare but for
// bf16 logits and masks, go by the lowest expert id. Selection thus compares the
// logits themselves: sigmoid and softmax keep their order, and two logits that
// a rounded score would merge still rank as they stand. -0 is turned into +0
// first, so that the two tie. What bounds the kernel is instructions (391 per
// token of 256 experts and eight places, one wave instruction in four clocks),
// not the logits' bytes: 8192 such tokens take 7.7 us, their 9.2 MB 1.5 us at the
// rate of a large copy; the gradient 8.0 us (387 instructions) for 18 MB. Both
// are near the time of the call itself (launch 1.6 us on the GPU, 6 us on the
// host). A token per wave is the plain form, not a measured optimum: four tokens
// of a wave in a 16-lane row each would share the maxima, four steps for four
// tokens, over lists four times as long. That is not built.
//
// Lane k then holds the k-th logit, and the weights of a token are computed in
// its lanes at once. All statistics are float; the renormalised weights come
// from exponentials of differences to the largest selected term, whose sum is
// at least 1.
//
// The gradient recomputes the softmax statistics from the logits (reading them
// is needed anyway, and it keeps nothing between the calls). With p the scores,
// d = scale * d_weights of the selected places:
//   softmax:  dx_e = p_e * ( [e selected] d_e - sum_k d_k p_k )
//   renorm:   dx_k = p_k * ( d_k - sum_j d_j p_j )   (sigmoid: times sigmoid(-x_k))
//   sigmoid:  dx_k = d_k * s_k * sigmoid(-x_k)
#include "experts.hpp"

namespace moe {
namespace {

constexpr uint32_t kKeyNegInf = 0x007fffffu;  // the keys of the infinities
constexpr uint32_t kKeyPosInf = 0xff800000u;

__device__ __forceinline__ float gate_load(const void *x, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(x)[i] << 16)
              : static_cast<const float *>(x)[i];
}
// A token's logits lane + 64 j, all loads in flight together (past the last
// expert the last one's again, which the callers leave out).
template <int V>
__device__ __forceinline__ void gate_row(const void *x, int64_t row, int E, bool bf16,
                                         float (&v)[V]) {
  const int lane = threadIdx.x & 63;
  if (bf16) {
    const uint16_t *p = static_cast<const uint16_t *>(x) + row;
#pragma unroll
    for (int j = 0; j < V; ++j)
      v[j] = __uint_as_float((uint32_t)p[min(lane + 64 * j, E - 1)] << 16);
  } else {
    const float *p = static_cast<const float *>(x) + row;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = p[min(lane + 64 * j, E - 1)];
  }
}

// Key of a selectable logit, 0 for -infinity; NaN and +infinity also give 0 and
// set bad. The keys of the finite floats are those between the infinities',
// which NaN of either sign fall outside of.
__device__ __forceinline__ uint32_t gate_key(float x, bool *bad) {
  const int32_t u = (int32_t)__float_as_uint(x + 0.0f);
  const uint32_t k = (uint32_t)(u ^ ((u >> 31) | (int32_t)0x80000000));
  const bool fin = k - (kKeyNegInf + 1u) < kKeyPosInf - (kKeyNegInf + 1u);
  *bad = *bad || (!fin && k != kKeyNegInf);
  return fin ? k : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {  // 0 -> -infinity
  const int32_t u = (int32_t)k;
  const float f = __uint_as_float((uint32_t)(u ^ (~(u >> 31) | (int32_t)0x80000000)));
  return k ? f : -INFINITY;
}

// exp(d) for d <= 0: the exponent d log2(e) is rounded once, so the result is off
// by 2^-24 |d| and one step. Only for a sum over all experts, where the terms of
// large |d| are small against the first, which is 1; the gradient, where a term
// is an expert's own result, takes expf.
__device__ __forceinline__ float exp_below(float d) {
  return __builtin_amdgcn_exp2f(d * 1.44269504f);
}

__device__ __forceinline__ float log_sigmoid(float x) {  // x may be -infinity
  return fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// The scores of lanes 0 .. K-1 (x = the lane's logit, -infinity where there is
// none); top and sum are the softmax statistics over all experts.
template <int kMode>
__device__ __forceinline__ float gate_score(float x, float top, float sum) {
  constexpr bool kSig = kMode & kGateSigmoid, kRenorm = kMode & kGateRenorm;
  float p;
  if (kRenorm) {
    const float z = kSig ? log_sigmoid(x) : x;
    // the largest term of the selected ones
    float m = z;
    for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float ez = x == -INFINITY ? 0.0f : expf(z - m);
    const float s = wave_sum_f(ez);
    p = x == -INFINITY ? 0.0f : ez / s;
  } else if (kSig) {
    p = x == -INFINITY ? 0.0f : sigmoid(x);
  } else {
    p = x == -INFINITY ? 0.0f : expf(x - top) / sum;
  }
  return p;
}

template <int V, int kMode>
__global__ __launch_bounds__(256) void gate_kernel(const void *__restrict__ x, int32_t T,
                                                   int32_t E, int32_t K, float scale, bool bf16,
                                                   int64_t *__restrict__ idx,
                                                   float *__restrict__ w, int32_t *status) {
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * (blockDim.x >> 6) +
                                                     (threadIdx.x >> 6)));
  if (t >= T) return;
  uint32_t key[V];
  bool bad = false;
  float logit[V];
  gate_row<V>(x, (int64_t)t * E, E, bf16, logit);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t k = gate_key(logit[j], &bad);
    key[j] = lane + 64 * j < E ? k : 0u;
  }
  uint32_t k0[V];
  int slot[V];  // the register a key came from
#pragma unroll
  for (int j = 0; j < V; ++j) {
    k0[j] = key[j];
    slot[j] = j;
  }
  constexpr bool kSorted = V <= 4;
  if (kSorted) {  // larger first, equal keys as they were
#pragma unroll
    for (int a = 0; a < V - 1; ++a)
#pragma unroll
      for (int b = 0; b < V - 1 - a; ++b) {
        const bool up = key[b + 1] > key[b];
        const uint32_t k1 = up ? key[b + 1] : key[b], k2 = up ? key[b] : key[b + 1];
        const int s1 = up ? slot[b + 1] : slot[b], s2 = up ? slot[b] : slot[b + 1];
        key[b] = k1;
        key[b + 1] = k2;
        slot[b] = s1;
        slot[b + 1] = s2;
      }
  }
  int my_id = -1;
  uint32_t my_key = 0, top_key = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t head = key[0];
    int at = slot[0];
    if (!kSorted) {
#pragma unroll
      for (int j = 1; j < V; ++j) {
        const bool up = key[j] > head;
        head = up ? key[j] : head;
        at = up ? j : at;
      }
    }
    const uint32_t m = wave_max_u(head);
    if (k == 0) top_key = m;
    if (m == 0) break;  // no selectable expert is left (uniform)
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
    if (lane == k) {
      my_id = id;
      my_key = m;
    }
    if (lane == l) {
      if (kSorted) {
#pragma unroll
        for (int j = 0; j + 1 < V; ++j) {
          key[j] = key[j + 1];
          slot[j] = slot[j + 1];
        }
        key[V - 1] = 0;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = j == at ? 0u : key[j];
      }
    }
  }
  // (a token without a selectable expert: every term is 0, no difference of infinities)
  const float top = top_key ? key_logit(top_key) : 0.0f;
  float sum = 1.0f;
  if (!(kMode & (kGateSigmoid | kGateRenorm))) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) s += exp_below(key_logit(k0[j]) - top);
    sum = wave_sum_f(s);
  }
  const float p = gate_score<kMode>(key_logit(my_key), top, sum);
  if (lane < K) {
    const int64_t o = (int64_t)t * K + lane;
    idx[o] = my_id;
    w[o] = my_id < 0 ? 0.0f : p * scale;
  }
  if (status && __ballot(bad) && lane == 0) atomicOr(status, kStBadLogit);
}

template <int V, int kMode>
__global__ __launch_bounds__(256) void gate_grad_kernel(
    const void *__restrict__ x, const int64_t *__restrict__ idx, const float *__restrict__ dw,
    int32_t T, int32_t E, int32_t K, float scale, bool bf16, void *__restrict__ dx,
    int32_t *status) {
  constexpr bool kSig = kMode & kGateSigmoid, kRenorm = kMode & kGateRenorm;
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * (blockDim.x >> 6) +
                                                     (threadIdx.x >> 6)));
  if (t >= T) return;
  constexpr bool kAll = !kSig && !kRenorm;  // softmax over all experts
  float logit[V];
  if (kAll) gate_row<V>(x, (int64_t)t * E, E, bf16, logit);
  int id = -1;
  float d = 0.0f, xs = -INFINITY;
  int st = 0;
  bool bad = false;
  if (lane < K) {
    const int64_t e = idx[(int64_t)t * K + lane];
    if (e >= 0 && e < E) {
      id = (int)e;
      d = dw[(int64_t)t * K + lane] * scale;
      xs = key_logit(gate_key(gate_load(x, (int64_t)t * E + id, bf16), &bad));
    } else if (e != -1) {
      st = kStBadExpert;
    }
  }
  if (xs == -INFINITY) id = -1;  // masked: contributes nothing
  float v[V], top = -INFINITY, sum = 1.0f;
  uint32_t key[V];
  if (kAll) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t k = gate_key(logit[j], &bad);
      key[j] = lane + 64 * j < E ? k : 0u;
      m = umax32(m, key[j]);
    }
    const uint32_t tk = wave_max_u(m);
    top = tk ? key_logit(tk) : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] = expf(key_logit(key[j]) - top);
      s += v[j];
    }
    sum = wave_sum_f(s);
  }
  const float p = gate_score<kMode>(xs, top, sum);
  float g;  // the gradient that lane k adds to its expert
  if (kAll) {
    g = id < 0 ? 0.0f : d * p;
    const float dot = wave_sum_f(g);
    const float r = sum > 0.0f ? dot / sum : 0.0f;
    // (a masked logit's 0 stays 0 where d_weights makes r infinite or NaN)
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = key[j] ? -v[j] * r : 0.0f;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.0f;
    g = id < 0 ? 0.0f : d;
    if (kRenorm) {
      const float dot = wave_sum_f(id < 0 ? 0.0f : d * p);
      g = id < 0 ? 0.0f : p * (d - dot);
    } else if (id >= 0) {
      g = d * p;
    }
    if (kSig && id >= 0) g *= sigmoid(-xs);
  }
  for (int k = 0; k < K; ++k) {  // the same expert twice adds up
    const int ik = __builtin_amdgcn_readlane(id, k);
    const float gk = lane_f(g, k);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += (ik == lane + 64 * j) ? gk : 0.0f;
  }
  if (bf16) {
    uint16_t *o = static_cast<uint16_t *>(dx) + (int64_t)t * E;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 64 * j < E) o[lane + 64 * j] = (uint16_t)ex_bf16(v[j]);
  } else {
    float *o = static_cast<float *>(dx) + (int64_t)t * E;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 64 * j < E) o[lane + 64 * j] = v[j];
  }
  const uint64_t be = __ballot(st != 0), bl = __ballot(bad);
  if (status && lane == 0 && (be | bl))
    atomicOr(status, (be ? kStBadExpert : 0) | (bl ? kStBadLogit : 0));
}

template <int V, int kMode>
hipError_t gate_vm(const void *x, int32_t T, int32_t E, int32_t K, bool bf16, float scale,
                   int64_t *idx, float *w, int32_t *status, hipStream_t s) {
  hipLaunchKernelGGL((gate_kernel<V, kMode>), dim3((unsigned)((T + 3) / 4)), dim3(256), 0, s, x, T,
                     E, K, scale, bf16, idx, w, status);
  return hipGetLastError();
}
template <int V, int kMode>
hipError_t gate_grad_vm(const void *x, const int64_t *idx, const float *dw, int32_t T, int32_t E,
                        int32_t K, bool bf16, float scale, void *dx, int32_t *status,
                        hipStream_t s) {
  hipLaunchKernelGGL((gate_grad_kernel<V, kMode>), dim3((unsigned)((T + 3) / 4)), dim3(256), 0, s,
                     x, idx, dw, T, E, K, scale, bf16, dx, status);
  return hipGetLastError();
}

}  // namespace

#define MOE_GATE_BY_V(FN, MODE, ...)                    \
  do {                                                  \
    if (E <= 64) return FN<1, MODE>(__VA_ARGS__);       \
    if (E <= 128) return FN<2, MODE>(__VA_ARGS__);      \
    if (E <= 256) return FN<4, MODE>(__VA_ARGS__);      \
    if (E <= 512) return FN<8, MODE>(__VA_ARGS__);      \
    return FN<16, MODE>(__VA_ARGS__);                   \
  } while (0)

hipError_t launch_gate(const void *x, int32_t T, int32_t E, int32_t K, int32_t flags, float scale,
                       int64_t *idx, float *w, int32_t *status, hipStream_t s) {
  const bool bf16 = flags & kGateBf16;
  switch (flags & (kGateSigmoid | kGateRenorm)) {
    case 0: MOE_GATE_BY_V(gate_vm, 0, x, T, E, K, bf16, scale, idx, w, status, s);
    case kGateSigmoid:
      MOE_GATE_BY_V(gate_vm, kGateSigmoid, x, T, E, K, bf16, scale, idx, w, status, s);
    case kGateRenorm:
      MOE_GATE_BY_V(gate_vm, kGateRenorm, x, T, E, K, bf16, scale, idx, w, status, s);
    default:
      MOE_GATE_BY_V(gate_vm, (kGateSigmoid | kGateRenorm), x, T, E, K, bf16, scale, idx, w, status,
                    s);
  }
}

hipError_t launch_gate_grad(const void *x, const int64_t *idx, const float *dw, int32_t T,
                            int32_t E, int32_t K, int32_t flags, float scale, void *dx,
                            int32_t *status, hipStream_t s) {
  const bool bf16 = flags & kGateBf16;
  switch (flags & (kGateSigmoid | kGateRenorm)) {
    case 0: MOE_GATE_BY_V(gate_grad_vm, 0, x, idx, dw, T, E, K, bf16, scale, dx, status, s);
    case kGateSigmoid:
      MOE_GATE_BY_V(gate_grad_vm, kGateSigmoid, x, idx, dw, T, E, K, bf16, scale, dx, status, s);
    case kGateRenorm:
      MOE_GATE_BY_V(gate_grad_vm, kGateRenorm, x, idx, dw, T, E, K, bf16, scale, dx, status, s);
    default:
      MOE_GATE_BY_V(gate_grad_vm, (kGateSigmoid | kGateRenorm), x, idx, dw, T, E, K, bf16, scale,
                    dx, status, s);
  }
}
#undef MOE_GATE_BY_V

}  // namespace moe
