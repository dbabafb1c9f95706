// Which kernel a product of the gated projection takes.  Plain C++, so that a test can
// ask on the CPU which of them its sizes reach.
#ifndef SILUQUANT_SWIGLU_PLAN_H
#define SILUQUANT_SWIGLU_PLAN_H

#include <stdint.h>

#include <algorithm>

namespace swiglu {

constexpr int kStageK = 64;  // values of k that a tile takes at once

// Which tiles a product of C [M, columns] over K takes (columns: the stored rows of B
// that it reads, 2H for the gated one), and in how many slices of K.
struct Plan {
  enum Tiles { k256, k128, k128Two, k64 } tiles;
  int slices;
};
// The times that decide are measured ones, in us: tiles of 256 x 256 take 1.0 a stage
// on an idle chip and 1.4 where every CU has one, and 7 for their ends; the others
// 0.5 to 0.58, 0.68 to 1.13 (two a CU) and 0.4 to 0.45.  Per kernel, all four measured
// (256, 128, 128 two a CU, 64 x 128): dx of 512 x 22016 x 4096 before slices 514, 200,
// 326, 153 us; dw of 22016 x 4096 x 1024 172, 225, 195 us; gated 777 x 1376 x 2048 44, 19,
// 25, 27 us, 300 x 1376 x 2048 44, 18.5, 24, 14.5 us.  The stages' times are those of
// loads into LDS; there is no term for bytes from memory, so that a few hundred rows of
// a wide weight are told too low: gated 64, 128, 256, 512 and 2048 rows of 11008 x 4096
// 29, 38, 65, 88 and 290 us where they take 45, 52, 80, 96 and 305.
static inline Plan plan(int64_t M, int64_t columns, int64_t K, bool by_k, bool sliced) {
  constexpr double kCus = 256;
  const double stages = (double)((K + kStageK - 1) / kStageK);
  Plan best = {Plan::k256, 1};
  double least = 1e300;
  // per_cu: workgroups at once; stage, full: us of a stage alone and what it takes more when every place is taken;
  // tile: us of a tile's ends
  auto look = [&](Plan::Tiles t, int tm, int tn, int per_cu, double stage, double full, double tile) {
    const double tiles = (double)((M + tm - 1) / tm) * (double)((columns + tn - 1) / tn);
    for (int slices = 1; slices <= (sliced ? 16 : 1); slices *= 2) {
      if (slices > 1 && (stages < 4 * slices || tiles * slices > per_cu * kCus)) break;
      const double busy = tiles * slices / (per_cu * kCus), rounds = __builtin_ceil(busy);
      double us = rounds * (__builtin_ceil(stages / slices) * (stage + full * std::min(1.0, busy)) + tile);
      if (slices > 1) us += 4.0 + (4.0 * slices + 4.0) * (double)M * (double)columns / 3e6;
      if (us < least) least = us, best = {t, slices};
    }
  };
  look(Plan::k256, 256, 256, 1, 1.0, 0.4, 7.0);
  look(Plan::k128, 128, 128, 1, 0.5, 0.08, 2.1);
  look(Plan::k128Two, 128, 128, 2, 0.68, 0.45, 2.0);
  if (!by_k) look(Plan::k64, 64, 128, 1, 0.4, 0.05, 1.5);
  return best;
}

// The gated product of M rows and N = H columns as a stream of the weight: the blocks
// of 16 rows that the kernel is for, 0 where it takes tiles.  The stream for up to 8
// rows, and up to 64 as long as tiles of 64 x 64 columns leave CUs without one.  In us,
// stream and tiles (H x D): 1 row of 11008 x 4096 36.7 and 41.4, 8 rows 41.2 and 41.6,
// 16 rows 46.2 and 41.8; 16 rows of 1376 x 2048 7.6 and 14.3, 32 rows 9.4 and 14.3, of
// 4096 x 4096 16.9 and 24.2, of 5504 x 2048 17.8 and 14.5; 48 rows of 1376 x 2048 12.2
// and 14.3, 64 rows of 4096 x 1024 8.2 and 9.4, of 2048 x 4096 24.0 and 24.3, of 5504 x
// 2048 26.6 and 14.5.
static inline int streamed(int64_t M, int64_t N, int64_t K) {
  if (!(M <= 8 || (M <= 16 && N <= 8192) || (M <= 32 && N <= 4096) || (M <= 64 && N <= 4096 && K <= 2048))) return 0;
  return M <= 16 ? 1 : M <= 32 ? 2 : 4;
}

}  // namespace swiglu

#endif
