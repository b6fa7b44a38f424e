// Host side of the tile products: choice of a geometry, grid sizes, launch.
#pragma once
#include <atomic>

#include "api_util.h"
#include "mm.h"

namespace moe {

using MMBig = MMGeom<256, 256, 4, 2, 64, 2, 2>;    // 8 waves, one block per CU
using MMMid = MMGeom<128, 128, 2, 2, 64, 2, 2>;    // 4 waves, two blocks per CU
using MMWide = MMGeom<64, 128, 2, 4, 64, 3, 4>;    // 8 waves, two blocks per CU
using MMSmall = MMGeom<64, 64, 2, 2, 64, 4, 2>;    // 4 waves, two blocks per CU

// What a geometry costs: rounds of resident blocks, each of `stage` us per 64-k
// stage plus `fixed` us for its first loads and its epilogue. Fitted to timings
// of NT products on one MI355X (us for Big / Mid / Wide / Small):
//   8192 x 4096 x 7168            372 / 462 / -   / -
//   4096 x 2048 x 1536             41 /  30 /  36 /  42
//   512 x 2048 x 768                - / 10.7 / 8.1 / 6.4
//   grouped, 128 experts, 32768 rows x 1536 x 2048   311 / 324 / 366 / 420
//   grouped, 128 experts,  4096 rows x 1536 x 2048   200 / 189 / 166 / 163
//   grouped, 14 of 128 experts, 16 rows x 1536 x 2048  30 / 22 / 15.7 / 17.2
struct MMCost {
  int bm, bn, slots;
  double stage, fixed;
};
constexpr MMCost kMMCost[4] = {{256, 256, 256, 1.60, 8.0},
                               {128, 128, 512, 1.00, 6.0},
                               {64, 128, 512, 0.62, 3.0},
                               {64, 64, 512, 0.36, 2.5}};

// m tiles of row blocks: of `rows` rows in one block (E = 0), or spread over E
// experts, where about half a tile per expert in use is left over and none has
// less than one.
inline double mm_row_tiles(int bm, int rows, int E) {
  if (E == 0) return (rows + bm - 1) / bm;
  const double act = rows < E ? rows : E, n = static_cast<double>(rows) / bm + 0.5 * act;
  return n > act ? n : act;
}
inline double mm_cost(const MMCost& c, double tiles, double stages) {
  const double rounds = tiles <= c.slots ? 1.0 : __builtin_ceil(tiles / c.slots);
  return rounds * (stages * c.stage + c.fixed);
}
// Index into kMMCost of the cheapest geometry for row-grouped products (NT, NN).
inline int mm_pick_rows(int rows, int E, int ndim, int kdim) {
  int best = 0;
  double at = 1e300;
  for (int i = 0; i < 4; ++i) {
    const MMCost& c = kMMCost[i];
    const double cost = mm_cost(c, mm_row_tiles(c.bm, rows, E) * ((ndim + c.bn - 1) / c.bn),
                                (kdim + 63) / 64);
    if (cost < at) {
      at = cost;
      best = i;
    }
  }
  return best;
}

template <class T, int MODE, class G>
hipError_t mm_launch(MMArgs a, hipStream_t s) {
  long long tiles;
  const bool swiglu = MODE == kModeNT && a.act == kActSwiglu;
  a.nt = swiglu ? (a.ndim / 2 + G::BN / 2 - 1) / (G::BN / 2) : (a.ndim + G::BN - 1) / G::BN;
  if (MODE == kModeTN) {
    a.mt = (a.mdim + G::BM - 1) / G::BM;
    tiles = static_cast<long long>(a.E) * a.splits * a.mt * a.nt;
  } else {
    // an upper bound over all ways to cut the rows: a partial tile per expert
    const long long partial = a.offsets ? (a.rows < a.E ? a.rows : a.E) : 1;
    tiles = (a.rows / G::BM + partial) * a.nt;
  }
  const long long grid = (tiles + 7) / 8 * 8;
  if (grid == 0) return hipSuccess;
  if (grid >= (1LL << 31)) return hipErrorInvalidConfiguration;
  // the attribute is set once per device (threads that race set it twice)
  static std::atomic<bool> ready[moe_api::kMaxDevices];
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= moe_api::kMaxDevices) return hipErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&mm_kernel<T, MODE, G>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, G::kLds);
    if (e != hipSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  hipLaunchKernelGGL((mm_kernel<T, MODE, G>), dim3(static_cast<unsigned>(grid)),
                     dim3(G::kThreads), G::kLds, s,
                     static_cast<const uint8_t*>(a.A), static_cast<const uint8_t*>(a.B), a);
  return hipGetLastError();
}

}  // namespace moe
