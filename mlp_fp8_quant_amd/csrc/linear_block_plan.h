// The kernel that fp8_linear_block runs for a shape (host code; a test asks it
// which shapes reach which kernel).
#pragma once

#include <stdint.h>

#include "kernels.h"

namespace fp8mot {

// How a shape runs (MI355X, 256 CUs; us measured).  Few outputs: the smallest
// tile whose grid gives no CU more than one workgroup: 1x4096x4096 5.3 with one
// block (with two 5.6), 64x4096x4096 7.6 with 32x32 (64x32 10.1, 32x16 10.6),
// 86x5351x1520 8.6 with 64x64 (64x32, two to some CUs, 11.3), 256x4096x4096 15.6 with
// 64x64 (128x64 18.0); and up to 64 rows 64x64 in pairs: 40x20000x4096 24.7 (128x64
// 35.8).
//
// More outputs: the least of the estimates below, rounds of workgroups times (rate
// * K + what a tile costs besides), the rate less where a round leaves CUs idle.
// Two K groups: 128x64 512x4096x12288 56 (128x128 67, 64x64 in pairs 77, 256x128
// 120) and 1024x2048x2048 12.7 (18.8, 15.8, 26), 128x128 2048x2048x8192 64 (128x64
// 75, without groups 68, 256x128 84).  Without: 128x64, three to a CU, 300x16384x2048
// 28.9 (128x128 32.0, with groups 36.8), 128x128, two, 5000x5000x4096 205 (128x64 218,
// 256x128 220), 256x128 4096x12288x4096 347 (128x128 357).
//
// The times above and the estimates are of W's scales for tiles and BF16 outputs.
// Of W's scales for rows, whose slots in LDS leave room for two workgroups of 128x64
// to a CU, the tiles take 6 to 19% longer, and the one chosen stays the best or
// within 4% of it: 4096x1536x2048 128x64 33.5 (256x128 34.2, 128x128 35.5; of tiles'
// scales 30.6, 32.4, 32.8), 5120x2048x1536 41.7 (53.3, 43.6), FP32 added in place 46.5
// (58.9, 48.2).
inline int linear_block_plan(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kCus = 256;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  auto one_each = [&](int64_t bm, int64_t bn) { return up(M, bm) * up(N, bn) <= kCus; };   // at most a tile per CU
  if (M <= 16) return one_each(16, 16) ? kRows1x1 : one_each(16, 32) ? kRows1x2 : kRows1x4;
  if (one_each(32, 16)) return kRows2x1;
  if (one_each(32, 32)) return kRows2x2;
  if (M <= 32) return kRows2x4;
  if (one_each(64, 32)) return kRows4x2;
  if (one_each(64, 64)) return kRows4x4;
  if (M <= 64) return kRows4x4Pair;
  const double k = (double)K;
  int best = kRows4x4Pair;
  double least = (double)up(up(M, 64) * up(N, 64), 2 * kCus) * (0.0056 * k + 4.6);
  auto offer = [&](int tile, double t) {
    if (t < least) {
      best = tile;
      least = t;
    }
  };
  const int64_t narrow = up(M, 128) * up(N, 64), square = up(M, 128) * up(N, 128), large = up(M, 256) * up(N, 128);
  if (narrow > INT32_MAX / 512) return kTile256x128;   // walks tiles: a launch counts its threads in 32 bits
  const double narrows = (double)narrow / kCus, pairs = (double)square / (2 * kCus);   // for each CU; pair of places
  auto fill = [&](int64_t tiles) { return tiles < kCus ? (double)tiles / kCus : 1.0; };
  offer(kTile128x64K2, (double)up(narrow, kCus) * ((0.0030 + 0.0012 * fill(narrow)) * k + 4.8));
  offer(kTile128x64, narrows <= 1.0   ? 0.0051 * k + 4.0
                     : narrows <= 2.0 ? (0.5 + 0.25 * narrows) * (0.0082 * k + 5.0)
                                      : narrows * (0.0044 * k + 0.9) + 3.0);
  offer(kTile128x128K2, (double)up(square, kCus) * ((0.0035 + 0.0032 * fill(square)) * k + 8.0));
  offer(kTile128x128, pairs <= 0.5 ? 0.0072 * k + 7.0
                                   : (pairs <= 1.0 ? 1.0 : 0.5 * (pairs + (double)up(square, 2 * kCus))) *
                                         (0.0128 * k + 7.0));
  offer(kTile256x128, (double)up(large, kCus) * (0.0118 * k + 9.0));
  return best;
}

}  // namespace fp8mot
