// What a workgroup needs to walk the rows of all segments when only the device
// knows the counts: the running sum of the experts' pieces in LDS.
#pragma once

#include <type_traits>

#include "experts.hpp"

namespace moe {

constexpr int kPlanThreads = 256;  // workgroup size of the stream kernels

struct SegmentPlan {
  int32_t first[kMaxExperts + 1];  // pieces of the experts before e; first[E] = all
  int32_t wave[16];
};
struct SegmentPlanRows : SegmentPlan {
  int32_t start[kMaxExperts];  // first buffer row of expert e
  uint8_t rows[kMaxExperts];   // its rows, for a kernel whose share has at most 255
};

// Cuts every segment into ceil(rows / piece) pieces and returns their number.
// Every thread of the workgroup (kThreads) must call it. Bad segments are
// reported by workgroup 0 alone.
template <int kThreads = kPlanThreads, class Plan>
__device__ __forceinline__ int plan_segments(const Segments &seg, int piece, Plan &p,
                                             int32_t *status) {
  constexpr int kMost = kMaxExperts / kThreads;
  const int per = (seg.E + kThreads - 1) / kThreads;  // consecutive experts per thread
  const int e0 = threadIdx.x * per;
  int n[kMost], mine = 0, coarse = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    n[i] = 0;
    if (i < per && e0 + i < seg.E) {
      int32_t st;
      bool ok;
      int r = segment_rows(seg, e0 + i, &st, &ok);
      coarse += (int)(((int64_t)r + 1023) >> 10);
      if (r <= seg.over || (seg.upto > 0 && r > seg.upto)) r = 0;
      if constexpr (std::is_same_v<Plan, SegmentPlanRows>) {
        p.start[e0 + i] = st;
        p.rows[e0 + i] = (uint8_t)r;
      }
      n[i] = (int)(((int64_t)r + piece - 1) / piece);
      bad = bad || !ok;
      mine += n[i];
    }
  }
  int total;
  if (seg.rows >= (1 << 20)) {
    // Segments that overlap against the rules could overflow the 32-bit sums
    // (up to 1024 segments of up to 2^31 rows): a coarse sum of all of them
    // first, in units of 1024 rows, and no pieces at all if it passes the
    // buffer's rows. What remains is less than 2^31 + 2^21.
    block_exclusive_scan(coarse, p.wave, kThreads / 64, &total);
    if ((uint32_t)total > (uint32_t)((seg.rows >> 10) + 1 + seg.E)) {
      mine = 0;
      bad = true;
#pragma unroll
      for (int i = 0; i < kMost; ++i) n[i] = 0;
    }
  }
  int at = block_exclusive_scan(mine, p.wave, kThreads / 64, &total);
  if (total < 0) {  // uniform: pieces of one row each past 2^31 - 1 after all
    total = at = 0;
    bad = true;
#pragma unroll
    for (int i = 0; i < kMost; ++i) n[i] = 0;
  }
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (i < per && e0 + i < seg.E) {
      p.first[e0 + i] = at;
      at += n[i];
    }
  }
  if (threadIdx.x == 0) p.first[seg.E] = total;
  if (bad && status && blockIdx.x == 0 && seg.over == 0) atomicOr(status, kStBadSlot);
  __syncthreads();
  return total;
}

// The expert of piece i, 0 <= i < first[E].
__device__ __forceinline__ int plan_find(const SegmentPlan &p, int E, int i) {
  int lo = 0, hi = E;  // first[lo] <= i < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.first[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace moe
