// Choice of geometry for the gradient products.
#pragma once
#include "mm_launch.h"

namespace moe {

// Tall: half of Big's work in a block of four waves, two blocks per CU, so that one
// block's loads and epilogue stand behind the other's multiplies. Both operands
// are M-major here, so stages of 32 rows still read whole cache lines. Slower than
// Big where there is much to multiply (8192 x 4096 from 7168 rows: 424 against
// 387 us), faster where a tile has few stages (128 experts x 1536 x 2048 from
// 32768 rows: 311 against 343 us; from 4096 rows: 159 against 207).
using MMTall = MMGeom<256, 128, 2, 2, 32, 2, 2>;
constexpr MMCost kMMTallCost = {256, 128, 512, 1.00, 1.20, 1.89, 5.4, 5.4};

// The geometry (0 Big, 1 Tall, 2 Mid, 3 Small) and the number of parts that an
// expert's rows are cut into: where the output tiles alone leave CUs idle the
// contraction is split, each part a float32 product in the workspace, added in
// order. A part costs its bytes: written, read, and the sum written, at about 4 TB/s.
struct TNPlan {
  int geom, splits;
  double cost;   // us
};
inline TNPlan mm_plan_tn(int rows, int E, int mdim, int ndim) {
  const MMCost* const table[4] = {&kMMBigCost, &kMMTallCost, &kMMMidCost, &kMMSmallCost};
  TNPlan best = {0, 1, 1e300};
  // ragged experts: half a stage is left over, and one with rows has at least one
  double stages = static_cast<double>(rows) / E / 64 + (E > 1 ? 0.5 : 0.0);
  if (stages < 1.0) stages = 1.0;
  const double out_bytes = 4.0 * E * mdim * ndim;
  for (int i = 0; i < 4; ++i) {
    const MMCost& c = *table[i];
    const double tiles = static_cast<double>(E) * ((mdim + c.bm - 1) / c.bm) *
                         ((ndim + c.bn - 1) / c.bn);
    for (int s = 1; s <= 32 && (s == 1 || stages >= 4.0 * s); s *= 2) {
      double cost = mm_cost(c, tiles * s, stages / s);
      if (s > 1) cost += 4.0 + out_bytes * (2 * s + 1) / 4e6;
      if (cost < best.cost) best = {i, s, cost};
    }
  }
  return best;
}

}  // namespace moe
