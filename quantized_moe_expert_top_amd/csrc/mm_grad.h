// Choice of geometry for the gradient products.
#pragma once
#include "mm_launch.h"

namespace moe {

// Tall: half of Big's work in a block of four waves, two blocks per CU, so that one
// block's loads and epilogue stand behind the other's multiplies. Both operands
// are M-major here, so stages of 32 rows still read whole cache lines. Slower than
// Big where there is much to multiply (8192 x 4096 from 7168 rows: 424 against
// 387 us), faster where a tile has few stages (128 experts x 1536 x 2048 from
// 32768 routed rows: 308 against 324 us; from 4096 rows, 32 each: 150 against 180).
using MMTall = MMGeom<256, 128, 2, 2, 32, 2, 2>;
constexpr MMCost kMMTallCost = {256, 128, 256, 512, 1.00, 1.20, 1.89, 5.4, 5.4, 5.4};

// A product's geometry and the number of parts that its contraction is cut into:
// where the output tiles alone leave CUs idle each part is a float32 product in the
// workspace, added in order. A part costs its bytes: written, read, and the sum
// written, at about 4 TB/s; `split_launch` stands for the sum's launch.
struct MMPlan {
  int geom, splits;
  double cost;   // us
};
constexpr double kMMSplitLaunch = 4.0;
inline double mm_split_cost(double values, int splits) {
  return splits > 1 ? 4.0 * values * (2 * splits + 1) / 4e6 : 0.0;
}
// The most parts (a power of two): each of four stages or more, and the parts' 64 x 64
// tiles at most kMMSplitTiles, a chip full several times over. So the parts of a call
// stay under 32 MB, and what the parts of up to `rows` rows take grows with rows:
// a workspace for the most rows serves fewer.
constexpr int kMMSplitTiles = 2048;
inline int mm_most_splits(double stages, double tiles64) {
  int s = 1;
  while (s < 32 && stages >= 8.0 * s && tiles64 * 2 * s <= kMMSplitTiles) s *= 2;
  return s;
}
inline double mm_tiles64(int a, int b) {
  return static_cast<double>((a + 63) / 64) * ((b + 63) / 64);
}
// 64-row stages of an expert's weight gradient; ragged experts: half a stage is left
// over, and one with rows has at least one
inline double mm_tn_stages(int rows, int E) {
  const double s = static_cast<double>(rows) / E / 64 + (E > 1 ? 0.5 : 0.0);
  return s < 1.0 ? 1.0 : s;
}
inline int mm_most_dw_splits(int rows, int E, int N, int K) {
  return mm_most_splits(mm_tn_stages(rows, E), E * mm_tiles64(N, K));
}
inline int mm_most_dx_splits(int rows, int N, int K) {
  return mm_most_splits((N + 63) / 64, mm_tiles64(rows, K));
}
// TN: 0 Big, 1 Tall, 2 Mid, 3 Small. Best with one part, or with several.
inline MMPlan mm_plan_tn(int rows, int E, int mdim, int ndim, bool split) {
  const MMCost* const table[4] = {&kMMBigCost, &kMMTallCost, &kMMMidCost, &kMMSmallCost};
  MMPlan best = {0, 1, 1e300};
  const double stages = mm_tn_stages(rows, E);
  const int most = split ? mm_most_dw_splits(rows, E, mdim, ndim) : 1;
  for (int i = 0; i < 4; ++i) {
    const MMCost& c = *table[i];
    const double tiles = static_cast<double>(E) * ((mdim + c.bm - 1) / c.bm) *
                         ((ndim + c.bn - 1) / c.bn);
    if (!mm_fits(static_cast<long long>(tiles) * most, c.threads)) continue;
    for (int s = split ? 2 : 1; s <= most; s *= 2) {
      const double cost = mm_cost(c, tiles * s, stages / s) +
                          mm_split_cost(static_cast<double>(E) * mdim * ndim, s);
      if (cost < best.cost) best = {i, s, cost};
    }
  }
  return best;
}
// NN without experts, in several parts: geometries of mm_pick_rows.
inline MMPlan mm_plan_nn_split(int rows, int ndim, int kdim) {
  const MMCost* const table[6] = {&kMMBigCost, &kMMMidCost, &kMMWideCost, &kMMSmallCost,
                                  &kMMLongCost, &kMMDeepCost};
  MMPlan best = {0, 1, 1e300};
  const double stages = (kdim + 63) / 64;
  const int most = mm_most_dx_splits(rows, kdim, ndim);
  for (int i = 0; i < 6; ++i) {
    const MMCost& c = *table[i];
    const double tiles = mm_row_tiles(c.bm, rows, 0) * ((ndim + c.bn - 1) / c.bn);
    for (int s = 2; s <= most; s *= 2) {
      const double cost = mm_cost(c, tiles * s, stages / s, true) +
                          mm_split_cost(static_cast<double>(rows) * ndim, s);
      if (cost < best.cost) best = {i, s, cost};
    }
  }
  return best;
}

}  // namespace moe
