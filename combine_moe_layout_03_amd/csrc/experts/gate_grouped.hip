// Router with a balance bias and groups: among the experts of the best groups
// the K largest choices c = score + bias of each token, and their weights, from
// the scores alone.
//
// Choices are compared as doubles: scores of different logits that a float would
// merge, or order wrongly by its rounding, still rank as they stand. Two kernels
// do that. One takes a token a wave and computes every choice in 64 bits; the
// other, for the usual shapes, takes four tokens a wave, orders floats and goes back
// to 64 bits only where two are too near to be told apart. 8192 tokens x 256 experts,
// 8 groups, top 8: 22 us by the first, 8.5 by the second, of which a launch is 1.6;
// bound by instructions (1155 for four tokens, at two waves a SIMD) and their
// latencies. Near choices cost little (one token in 100 has some among its best, one
// in 8000 two groups on the border), a token that is done again 4 us at the call's
// end. 16 tokens: 9.2 and 4.8 us.
#include "gate.hpp"

#include <type_traits>

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

// The high words' maximum, then the low ones' among those that have it.
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t m) {
  const uint32_t hi = wave_max_u((uint32_t)(m >> 32));
  const uint32_t lo = wave_max_u((uint32_t)(m >> 32) == hi ? (uint32_t)m : 0u);
  return (uint64_t)hi << 32 | lo;
}
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, 0xf, 0xf, false);
}
template <int kCtrl>
__device__ __forceinline__ double dpp_d(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return __longlong_as_double((int64_t)((uint64_t)dpp_u<kCtrl>((uint32_t)u) |
                                        (uint64_t)dpp_u<kCtrl>((uint32_t)(u >> 32)) << 32));
}
__device__ __forceinline__ double lane_d(double x, int lane) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return __longlong_as_double(
      (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane) |
                (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane)
                    << 32));
}
__device__ __forceinline__ double wave_sum_d(double x) {
  x += dpp_d<0x128>(x);
  x += dpp_d<0x124>(x);
  x += dpp_d<0x122>(x);
  x += dpp_d<0x121>(x);
  return (lane_d(x, 0) + lane_d(x, 16)) + (lane_d(x, 32) + lane_d(x, 48));
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

// One token, in one wave: expert e = lane + 64 * j in register j. Its choice is the
// logit itself without a bias (as moe_gate compares), else score + bias as a double.
// `choices` is LDS of 64 V keys of the wave's own.
template <int V, int kMode>
__device__ void exact_token(const GroupArgs &a, int t, uint64_t *choices, bool *bad) {
  constexpr bool kSig = kMode & kGateSigmoid;
  const int lane = threadIdx.x & 63;
  const int E = a.E;
  float x[V];
  gate_row<V>(a.x, (int64_t)t * E, E, a.bf16, x);
  uint64_t key[V];
  uint32_t top_key = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t k = gate_key(x[j], bad);
    x[j] = lane + 64 * j < E && k ? key_logit(k) : -INFINITY;
    top_key = umax32(top_key, lane + 64 * j < E ? k : 0u);
  }
  top_key = wave_max_u(top_key);
  const float top = top_key ? key_logit(top_key) : 0.0f;
  const bool scores = a.bias || (a.sum2 && a.G > 1) || !(kMode & (kGateSigmoid | kGateRenorm));
  double sum = 1.0;
  double p[V];
  if (scores) {
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
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    bool ok = x[j] != -INFINITY;
    double c = x[j];
    if (a.bias) {
      const float b = a.bias[min(lane + 64 * j, E - 1)];
      if (gate_key(b, bad) == 0) ok = false;
      c = p[j] + (double)b;
    }
    key[j] = ok ? choice_key(c) : kNone;
  }
  if (a.G > 1) {
    const int n = E / a.G;
    const bool by_score = a.sum2 && !a.bias;  // the groups' keys differ from the choices'
#pragma unroll
    for (int j = 0; j < V; ++j)
      choices[lane + 64 * j] = by_score && key[j] != kNone ? choice_key(p[j]) : key[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    // lane g: group g
    uint64_t group = kNone;
    if (lane < a.G) {
      uint64_t k1 = kNone, k2 = kNone;
#pragma unroll 8
      for (int i = 0; i < n; ++i) {
        const uint64_t k = choices[lane * n + i];
        const uint64_t lo = k < k1 ? k : k1;
        k1 = k > k1 ? k : k1;
        k2 = lo > k2 ? lo : k2;
      }
      group = k1;
      if (a.sum2 && k2 != kNone) group = choice_key(key_choice(k1) + key_choice(k2));
    }
    __builtin_amdgcn_wave_barrier();
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
}

template <int V, int kMode>
__global__ __launch_bounds__(256) void gate_grouped_kernel(GroupArgs a) {
  __shared__ uint64_t choices[4][V * 64];
  const int wave = threadIdx.x >> 6;
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + wave));
  if (t >= a.T) return;
  bool bad = false;
  exact_token<V, kMode>(a, t, choices[wave], &bad);
  if (a.status && __ballot(bad) && (threadIdx.x & 63) == 0) atomicOr(a.status, kStBadLogit);
}

// ---- four tokens a wave -----------------------------------------------------------
//
// A token has the 16 lanes of a DPP row, lane c the experts c V ... c V + V - 1, so that
// maxima over a token's lanes are four steps for four tokens, and a group is a run of
// L lanes. Choices are floats here, and their keys give up their lowest bits to the
// expert's place in its lane. That orders all but neighbours closer than `near`: the
// exact order of those is settled among the token's 16 best candidates, one a
// lane, by their doubles, and of groups by their best two's; where that does not reach
// (more candidates or groups within reach, a softmax's sum in doubt) the token is done
// again by exact_token.

__device__ __forceinline__ float row_sum16(float x) {
  x += dpp_f<0x128>(x);
  x += dpp_f<0x124>(x);
  x += dpp_f<0x122>(x);
  return x + dpp_f<0x121>(x);
}
__device__ __forceinline__ float row_max16(float x) {
  x = fmaxf(x, dpp_f<0x128>(x));
  x = fmaxf(x, dpp_f<0x124>(x));
  x = fmaxf(x, dpp_f<0x122>(x));
  return fmaxf(x, dpp_f<0x121>(x));
}

// How close two choices, rounded and without the places in their keys, may be to
// be told apart: 2^-21 for a score (its exponential's argument and result, the sum
// and the quotient, at slopes of at most 1/4; a softmax's sum of 256 terms is common
// to both), 2^-24 of the sum with the bias, 2^-19 for the place, twice each and
// twice that. Logits are as they stand: equal but for the places.
__device__ __forceinline__ float near(float c, bool exact, float largest_score) {
  return exact ? 0.0f : 0x1p-18f * largest_score + 0x1p-17f * fabsf(c);
}

// The best two of the L lanes of a group, in all of them.
template <int kCtrl>
__device__ __forceinline__ void best_two(float &m1, float &m2) {
  const float o1 = dpp_f<kCtrl>(m1), o2 = dpp_f<kCtrl>(m2);
  m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
  m1 = fmaxf(m1, o1);
}

// How many groups of the row score more than the lane's for sure, and how many may: by
// more than the two scores may be off together (tol is each group's own), and by more
// than less that. Of equal ones the first scores more.
template <int L, int kStart = L>
__device__ __forceinline__ void better_groups(float s, float tol, int &sure, int &maybe) {
  if constexpr (kStart < 16) {
    const float o = dpp_f<0x120 + kStart>(s);  // of lane c - kStart, around the row
    const float both = tol + dpp_f<0x120 + kStart>(tol);
    const bool first = (int)(threadIdx.x & 15) >= kStart;
    sure += (o > s + both) | (first & (o == s + both));
    maybe += (o > s - both) | (first & (o == s - both));
    better_groups<L, kStart + L>(s, tol, sure, maybe);
  }
}

template <int kCtrl>
__device__ __forceinline__ void best_two_d(double &m1, double &m2) {
  const double o1 = dpp_d<kCtrl>(m1), o2 = dpp_d<kCtrl>(m2);
  m2 = fmax(fmin(m1, o1), fmax(m2, o2));
  m1 = fmax(m1, o1);
}

// How many groups score more than the lane's, those too near by their doubles.
template <int L, int kStart = L>
__device__ __forceinline__ void settle_groups(float s, float tol, double sd, bool unsure,
                                              int &better, bool &open) {
  if constexpr (kStart < 16) {
    const float o = dpp_f<0x120 + kStart>(s);
    const float both = tol + dpp_f<0x120 + kStart>(tol);
    const double od = dpp_d<0x120 + kStart>(sd);
    const bool known = dpp_u<0x120 + kStart>(unsure) != 0u;
    const bool first = (int)(threadIdx.x & 15) >= kStart;
    const bool near = !(o > s + both) && !(o < s - both);
    open |= near & !known;
    better += near ? (od > sd) | (first & (od == sd)) : o > s + both;
    settle_groups<L, kStart + L>(s, tol, sd, unsure, better, open);
  }
}

__device__ __forceinline__ uint32_t float_key(float x) {
  const int32_t u = (int32_t)__float_as_uint(x);
  return (uint32_t)(u ^ ((u >> 31) | (int32_t)0x80000000));
}

// Larger keys first (Batcher's odd-even merges).
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j <= V - 1 - q; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t lo = k[i + j] < k[i + j + q] ? k[i + j] : k[i + j + q];
            k[i + j] = umax32(k[i + j], k[i + j + q]);
            k[i + j + q] = lo;
          }
}

// How many of the row's 16 candidates come before the lane's. A softmax's choices
// rest on a float sum, off by 2^-19 of it at most (16 + 4 additions and the terms'
// own errors), which moves two choices apart by as much of the scores' difference:
// doubt, where that decides. (Equal logits have equal scores whatever the sum.)
template <bool kDoubt, int kStart = 1>
__device__ __forceinline__ int better_candidates(double c, float p, float x, uint32_t id,
                                                 bool &doubt) {
  if constexpr (kStart >= 16) {
    return 0;
  } else {
    const double o = dpp_d<0x120 + kStart>(c);
    const uint32_t oid = dpp_u<0x120 + kStart>(id);
    if (kDoubt) {
      const float op = dpp_f<0x120 + kStart>(p);
      const bool same = dpp_f<0x120 + kStart>(x) == x;
      doubt |= !same & (fabs(o - c) <= (double)(0x1p-18f * (fabsf(op - p) + 0x1p-22f * p)));
    }
    return (o > c || (o == c && oid < id)) +
           better_candidates<kDoubt, kStart + 1>(c, p, x, id, doubt);
  }
}

// NaN or +infinity
__device__ __forceinline__ bool wrong(float x) {
  return __builtin_amdgcn_classf(x, 0x001 | 0x002 | 0x200);
}

template <int V, int kMode>
__global__ __launch_bounds__(256) void gate_rows_kernel(GroupArgs a, int lanes) {
  constexpr bool kSig = kMode & kGateSigmoid, kRenorm = kMode & kGateRenorm;
  constexpr int kExact = (V * 16 + 63) / 64;  // registers of a token in a whole wave
  constexpr uint32_t kPlace = V > 8 ? 15 : V > 4 ? 7 : 3;
  __shared__ uint64_t choices[4][kExact * 64];
  __shared__ ex_u32x2 taken[4][64];  // a lane's key and the lane, in order
  const int lane = threadIdx.x & 63, c = lane & 15, wave = threadIdx.x >> 6;
  const int t0 = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + wave)) * 4;
  if (t0 >= a.T) return;
  const int t = t0 + (lane >> 4), tt = min(t, a.T - 1);
  const int E = a.E, K = a.K;
  const int64_t row = (int64_t)tt * E;
  bool bad = false;
  float x[V], v[V];
  if (a.bf16) {
    uint32_t w[V / 2];
    __builtin_memcpy(w, static_cast<const uint16_t *>(a.x) + row + c * V, V * 2);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      x[2 * j] = ex_lo(w[j]);
      x[2 * j + 1] = ex_hi(w[j]);
    }
  } else {
    __builtin_memcpy(x, static_cast<const float *>(a.x) + row + c * V, V * 4);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    bad |= wrong(x[j]);
    x[j] = __builtin_isfinite(x[j]) ? x[j] + 0.0f : -INFINITY;
    v[j] = x[j];
  }
  const bool sums = a.sum2 && a.G > 1, exact = !a.bias;
  float top = 0.0f, sum = 1.0f;
  if (!kSig && (!kRenorm || a.bias || sums)) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, x[j]);
    m = row_max16(m);
    top = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) s += exp_below(x[j] - top);
    sum = row_sum16(s);
  }
  const float largest = kSig ? 1.0f : 1.0f / sum;  // no score is larger
  float g1 = -INFINITY, g2 = -INFINITY;  // the lane's best two choices, for its group
  float by[V];                           // what its group is scored by
#pragma unroll
  for (int j = 0; j < V; ++j) by[j] = x[j];
  if (a.bias || sums) {
    float b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = 0.0f;
    if (a.bias) __builtin_memcpy(b, a.bias + c * V, V * 4);
    const float r = kSig ? 1.0f : __builtin_amdgcn_rcpf(sum);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float s = kSig ? __builtin_amdgcn_rcpf(
                                 1.0f + __builtin_amdgcn_exp2f(x[j] * -1.44269504f))
                           : exp_below(x[j] - top) * r;
      bad |= wrong(b[j]);
      // (one masked by its logit or bias)
      const float choice = __builtin_isfinite(x[j] + b[j] * 0.0f) ? s + b[j] : -INFINITY;
      g2 = __builtin_amdgcn_fmed3f(g1, g2, choice);
      g1 = fmaxf(g1, choice);
      by[j] = choice;
      v[j] = a.bias ? choice : x[j];
    }
  } else if (a.G > 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) g1 = fmaxf(g1, x[j]);
  }
  bool unsure = false;
  bool kept = true;
  if (a.G > 1) {  // so a group has 1, 2, 4 or 8 lanes
    if (lanes > 1) best_two<0xB1>(g1, g2);
    if (lanes > 2) best_two<0x4E>(g1, g2);
    if (lanes > 4) best_two<0x141>(g1, g2);
    // Choices are compared as quarters, so that neither the sum of two nor a tolerance
    // beside it passes the float range; logits as they stand.
    const bool chosen = a.bias || sums;
    float s = g1;
    if (chosen) s = 0.25f * g1 + (sums && g2 != -INFINITY ? 0.25f * g2 : 0.0f);
    // How far a group's score may be off: each of its two scores by 2^-21; by 2^-24 of
    // each choice, which may cancel in their sum, and as much again for the sum and for
    // the comparison. A softmax's common sum, off by 2^-19 of it, moves two groups apart by
    // as much of the difference of their scores, which biases may make up for: twice the
    // largest score at most, half of it on each side.
    const float e1 = fabsf(g1), e2 = sums && g2 != -INFINITY ? fabsf(g2) : 0.0f;
    const float tol = !chosen || s == -INFINITY
                          ? 0.0f
                          : 0.25f * (kSig ? 0x1p-20f : 0x1.8p-19f) * largest +
                                (0x1p-24f * e1 + 0x1p-24f * e2);
    int sure = 0, maybe = 0;
    switch (lanes) {
      case 1: better_groups<1>(s, tol, sure, maybe); break;
      case 2: better_groups<2>(s, tol, sure, maybe); break;
      case 4: better_groups<4>(s, tol, sure, maybe); break;
      default: better_groups<8>(s, tol, sure, maybe);
    }
    kept = sure < a.KG;
    unsure = kept && maybe >= a.KG;
    if (kSig && __ballot(unsure)) {  // uniform, and rare: the groups on the border in 64 bits
      // Of a group that is unsure, the choices that may be its best two: those as near to
      // the last of them as two choices may be off.
      const float edge = sums ? g2 : g1, least = edge - (0x1p-18f + 0x1p-20f * fabsf(edge));
      double d1 = -INFINITY, d2 = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = unsure && by[j] != -INFINITY && !(by[j] < least);
        if (!__ballot(in)) continue;
        double d = 1.0 / (1.0 + exp(-(double)x[j]));
        if (a.bias) d += (double)a.bias[c * V + j];
        if (!in) d = -INFINITY;
        d2 = fmax(d2, fmin(d1, d));
        d1 = fmax(d1, d);
      }
      if (lanes > 1) best_two_d<0xB1>(d1, d2);
      if (lanes > 2) best_two_d<0x4E>(d1, d2);
      if (lanes > 4) best_two_d<0x141>(d1, d2);
      const double sd = sums && d2 != -INFINITY ? d1 + d2 : d1;
      int better = 0;
      bool open = false;  // one as near that has no such value
      switch (lanes) {
        case 1: settle_groups<1>(s, tol, sd, unsure, better, open); break;
        case 2: settle_groups<2>(s, tol, sd, unsure, better, open); break;
        case 4: settle_groups<4>(s, tol, sd, unsure, better, open); break;
        default: settle_groups<8>(s, tol, sd, unsure, better, open);
      }
      if (unsure) {
        kept = better < a.KG;
        unsure = open;
      }
    }
  }
  // A masked expert's key is that of -infinity, an exhausted list's or dropped
  // group's head 0.
  uint32_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = (float_key(v[j]) & ~kPlace) | (kPlace - j);
  sort_keys<V>(key);
  key[0] = kept ? key[0] : 0u;
  constexpr int kShort = V < 9 ? V : 9;  // of a list, for up to eight places
  auto take = [&](int k, auto depth) {   // the k-th candidate
    const uint32_t m = row16_max(key[0]);
    // of equal choices the first lane's, so the lower id
    const uint64_t same = __ballot((key[0] ^ m) <= kPlace);
    const int first = __ffs((int)((uint32_t)(same >> (lane & 48)) & 0xffffu)) - 1;
    if (c == first && m) {
      taken[wave][lane & 48 | k] = ex_u32x2{key[0], (uint32_t)lane};
#pragma unroll
      for (int j = 0; j + 1 < depth.value; ++j) key[j] = key[j + 1];
      key[depth.value - 1] = 0u;
    }
  };
  taken[wave][lane] = ex_u32x2{0u, 0u};
  if (K <= 8) {
    for (int k = 0; k <= K; ++k) take(k, std::integral_constant<int, kShort>{});
  } else {
    for (int k = 0; k <= K; ++k) take(k, std::integral_constant<int, V>{});
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  uint32_t my_key = taken[wave][lane].x;
  int my_lane = (int)taken[wave][lane].y & 15;
  my_key = my_key > kKeyNegInf ? my_key : 0u;
  auto value = [&](uint32_t k) {  // of a key without its place
    const int32_t u = (int32_t)(k & ~kPlace);
    return __uint_as_float((uint32_t)(u ^ (~(u >> 31) | (int32_t)0x80000000)));
  };
  int place = c;  // where the lane's candidate stands
  const uint32_t before = dpp_u<0x111>(my_key);
  const float f = value(my_key);
  // (equal bf16 logits are in order; others with equal keys may differ in the places)
  const bool tie = c >= 1 && c <= K && my_key && value(before) - f <= near(f, exact, largest) &&
                   !(exact && a.bf16);
  if (__ballot(tie)) {  // uniform
    const uint64_t rows = __ballot(tie);
    const bool here = (uint32_t)(rows >> (lane & 48)) & 0xffffu;
    for (int k = K + 1; k < 16; ++k) take(k, std::integral_constant<int, V>{});
    // a short list that ended may have had more
    if (K <= 8 && V > kShort && here && kept && key[0] == 0u) unsure = true;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    my_key = taken[wave][lane].x;
    my_lane = (int)taken[wave][lane].y & 15;
    my_key = my_key > kKeyNegInf ? my_key : 0u;
    const int id = my_key ? my_lane * V + (int)(kPlace - (my_key & kPlace)) : E + c;
    const float xc = gate_load(a.x, row + min(id, E - 1), a.bf16);
    double d = xc;
    float score = 0.0f;
    if (a.bias) {
      const double e = exp(kSig ? -(double)xc : (double)xc - (double)top);
      d = kSig ? 1.0 / (1.0 + e) : e / (double)sum;
      score = (float)d;
      d += (double)a.bias[min(id, E - 1)];
    }
    if (!my_key) d = -INFINITY;
    bool doubt = false;
    const int rank = better_candidates<!kSig>(d, score, xc, (uint32_t)id, doubt);
    unsure |= here && doubt && !exact;
    if (here) {
      place = rank;
      // the last candidate bounds those that are none
      const uint32_t last = (uint32_t)__shfl((int)my_key, (lane & 48) + 15);
      if (rank == K - 1 && my_key && last && value(my_key) - value(last) <= near(value(last), exact, largest))
        unsure = true;
    }
  }
  const uint64_t again = __ballot(unsure);
  const bool on = place < K, found = on && my_key;
  const int id = found ? my_lane * V + (int)(kPlace - (my_key & kPlace)) : -1;
  float xs = -INFINITY;
  if (found) xs = gate_load(a.x, row + id, a.bf16);
  float p;
  if (kRenorm) {
    const float z = kSig ? log_sigmoid(xs) : xs;
    const float m = row_max16(found ? z : -INFINITY);
    const float ez = found ? expf(z - m) : 0.0f;
    const float all = row_sum16(ez);
    p = found ? ez / all : 0.0f;
  } else if (kSig) {
    p = found ? sigmoid(xs) : 0.0f;
  } else {
    p = found ? expf(xs - top) / sum : 0.0f;
  }
  if (on && t < a.T && !((uint32_t)(again >> (lane & 48)) & 0xffffu)) {
    const int64_t o = (int64_t)t * K + place;
    a.idx[o] = id;
    a.w[o] = found ? p * a.scale : 0.0f;
  }
  if (again) {  // uniform
#pragma unroll 1
    for (int r = 0; r < 4; ++r)
      if ((again >> (16 * r) & 0xffff) && t0 + r < a.T)
        exact_token<kExact, kMode>(a, t0 + r, choices[wave], &bad);
  }
  if (a.status && __ballot(bad) && lane == 0) atomicOr(a.status, kStBadLogit);
}

template <int V, int kMode>
hipError_t gate_grouped_vm(const GroupArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((gate_grouped_kernel<V, kMode>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0,
                     s, a);
  return hipGetLastError();
}
template <int V, int kMode>
hipError_t gate_rows_vm(const GroupArgs &a, int lanes, hipStream_t s) {
  hipLaunchKernelGGL((gate_rows_kernel<V, kMode>), dim3((unsigned)((a.T + 15) / 16)), dim3(256), 0,
                     s, a, lanes);
  return hipGetLastError();
}

// Lanes of a group where a token fits a row of 16: an even number of experts a lane
// (whole words of bf16), at most 16 (the places in a key), K + 1 candidates, groups of
// whole lanes whose number is a power of two, rows on whole words. 0: a wave a token.
// 8192 tokens, us, four a wave and one: 32 experts 5.6 and 10.7, 64 6.4 and 12.2, 96 6.8
// and 15.8, 128 7.1 and 16.1, 160 7.5 and 20.6, 192 7.7 and 21.7, 224 8.2 and 22.3, 256 8.5
// and 22.1; 16 tokens x 256 4.8 and 9.2. More experts, one token a wave: 320 33, 512 36.
int row_lanes(const GroupArgs &a) {
  const int v = a.E / 16, n = a.E / a.G;
  if (a.E % 32 || v > 16 || a.K > 15 || n % v) return 0;
  if (reinterpret_cast<uintptr_t>(a.x) & 3u) return 0;
  const int lanes = n / v;
  return lanes & (lanes - 1) ? 0 : lanes;
}

template <int kMode>
hipError_t gate_grouped_m(const GroupArgs &a, hipStream_t s) {
  if (const int lanes = row_lanes(a)) {
    switch (a.E / 16) {
      case 2: return gate_rows_vm<2, kMode>(a, lanes, s);
      case 4: return gate_rows_vm<4, kMode>(a, lanes, s);
      case 6: return gate_rows_vm<6, kMode>(a, lanes, s);
      case 8: return gate_rows_vm<8, kMode>(a, lanes, s);
      case 10: return gate_rows_vm<10, kMode>(a, lanes, s);
      case 12: return gate_rows_vm<12, kMode>(a, lanes, s);
      case 14: return gate_rows_vm<14, kMode>(a, lanes, s);
      default: return gate_rows_vm<16, kMode>(a, lanes, s);
    }
  }
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
