// Which kernel a dense product takes: arithmetic on its sizes alone, in plain C++.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kStep = 64;  // k of a stage: 128 bytes of a row

struct Plan {
  int high, wide;     // fragments of 16 a wave has: tiles of 32 high x 32 wide
  int splits, steps;  // parts of k and their stages
};

// The tile whose rounds over the 256 CUs take the least, in units of 22 ns, what a
// wave takes for a fragment's products of a stage; starting and storing a tile takes
// about 11 us, eight stages of a large one. (8192 x 7168 columns in rounds of 3.5
// tiles of 256: 229 us, of 4 tiles of 224 wide: 207; 8192 x 2048 the other way round,
// 180 against 279.) The partial sums of a split one stay within `workspace` bytes.
inline Plan plan(int64_t rows, int64_t cols, int64_t k, bool pairs, int64_t workspace) {
  const int64_t steps = (k + kStep - 1) / kStep;
  auto tiles = [&](int64_t h, int64_t w) {
    return ((rows + 32 * h - 1) / (32 * h)) * ((cols + 32 * w - 1) / (32 * w));
  };
  Plan p{8, 8, 1, (int)steps};
  double best = 0;
  for (int w = 8; w >= 6; w -= pairs ? 2 : 1) {  // (a wave has both halves of its pairs)
    const double t = (double)((tiles(8, w) + 255) / 256) * (8 * w * steps + 520);
    if (w == 8 || t < best) {
      best = t;
      p.wide = w;
    }
  }
  // Small tiles, two to a CU: half a microsecond a stage alone, 0.8 beside another;
  // a large one's stage takes 1.4. Parts of k, written and read again, only
  // where there are tiles for at most half the CUs.
  const int64_t n = tiles(4, 4), last = n % 512;
  const double small = (double)(n / 512) * (38 * steps + 364) +
                       (last == 0 ? 0.0 : last <= 256 ? 23 * steps + 180 : 38 * steps + 364);
  if (best <= small) return p;
  p.high = p.wide = 4;
  int64_t s = 256 / n;
  if (s > steps / 8) s = steps / 8;
  const int64_t fit = workspace / 4 / (rows * cols);
  if (s > fit) s = fit;
  if (s > 1) {
    p.steps = (int)((steps + s - 1) / s);
    p.splits = (int)((steps + p.steps - 1) / p.steps);
  }
  return p;
}

// Whether a product is streamed, its rows in blocks of 16 that each read the weights
// again: with one block of 1024 channels or more always; else where its units of 16 x 16
// are at most 1024 (two rounds of two to a CU) and what they read is at most 3.7 million
// channels of 32 rows. Streamed against tiles, us: 1024 units of 256 channels 5.2 and 6.4,
// 2048 of them 8.9 and 6.6; 1024 units of 512 or 2048 channels 5.9 and 8.2, 10.4 and 12.6;
// 768 of 4096 14.9 and 16.4, 1024 of them 18.6 to 21 and 17.4; 512 of 7168 16 to 20 and 18
// to 20, 640 of them 23 and 20; 16 rows x 65536 of 256 or 512 channels 20 and 11, 24 and 18,
// 16 x 32768 of 2048: 27 and 36. (Of several blocks with long sums neither side is near
// its operands' bytes: 128 x 1024 of 7168 is 17 MB, 3 us.) The second half of a SwiGLU's
// weights has to be within reach of a 32-bit offset.
inline bool streamed(int64_t rows, int64_t N, int64_t k, bool pairs) {
  if (pairs && (N + 16) * k * 2 >= 0xffffffe0ll) return false;
  const int64_t units = (rows + 15) / 16 * ((N * (pairs ? 2 : 1) + 15) / 16);
  return (rows <= 16 && k >= 1024) || (units <= 1024 && units * k <= 3700000);
}

// Eight weight rows a workgroup where that is one for every CU at most (7168 channels, 16
// rows x 256: 7.8 against 10.1 us, 128 x 256: 7.0 against 8.1, 16 x 2048: 9.5 against 11.1;
// 16 x 2304, 128 x 288, where it is not, 14.9 against 11.3 and 9.9 against 8.0).
inline int stream_weight_rows(int64_t rows, int64_t N, bool pairs) {
  const int64_t w = pairs ? 2 * N : N;
  return (rows + 15) / 16 * ((w + 7) / 8) <= 256 ? 8 : 16;
}

}  // namespace moe
