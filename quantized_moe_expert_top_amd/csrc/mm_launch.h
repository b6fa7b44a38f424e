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
// 4 waves, two blocks per CU: one block's loads and epilogue stand behind the
// other's multiplies. Its 32-k stages read half cache lines of a K-major operand,
// so a long K goes to Big (8192 x 4096 x 7168: 447 us expected against 376). With few
// stages it is level or ahead (routed rows of 128 experts, 8 to 1513 of 32768 each:
// 2048 x 768 to float32 225 us, Big 226; its row gradient 164, Big 171; row gradient
// of 1536 x 2048 288, Big 297; behind where every expert has 256: 253, Big 233, which
// the host cannot see). Waves of 128 x 64 (of 64 x 128: 226 and 291 for 225 and 288).
using MMLong = MMGeom<128, 256, 1, 4, 32, 3, 2>;
// 8 waves, one block per CU, four stages: where a dense product has too few tiles
// for two blocks per CU a block alone has to keep enough loads in flight (1219 x 1728
// x 5120: 40 us, Mid 60, Wide 50; 5549 x 384 x 5760: 40, Mid 63, Wide 53).
using MMDeep = MMGeom<128, 128, 2, 4, 64, 4, 2>;

// What a geometry costs, in us on one MI355X: a round of resident blocks takes
// `s1`, `s2` or `s3` per 64-k stage with 64, 256 or `slots` blocks at work (fewer
// blocks, more of the caches' rate for each), and `full` (a full round with experts'
// weights from memory; `dense` without) or `part` (the last round) for first loads
// and epilogues. Fitted; what the fit says and, in brackets, what was timed
// (cards differ by up to 7%):
//   NT  8192 x 4096 x 7168   Big 395 (376)   Mid 460 (462)
//       4096 x 2048 x 1536   Big 40 (44)     Mid 31 (31)    Wide 36 (35)    Small 45 (42)
//       6115 x 5728 x 176    Big 46 (51)     Mid 46 (42)    Wide 39 (34)    Small 53 (51)
//       5549 x 384 x 5760    Big 110 (115)   Mid 62 (64)    Wide 55 (55)    Small 59 (55)
//       512 x 2048 x 768     Mid 11 (10.7)   Wide 7.6 (8.1) Small 6.3 (6.5)
//       grouped, 128 experts, 32768 x 1536 x 2048   Big 297 (306)   Mid 302 (320)
//       grouped, 128 experts, 32768 x 2048 x 768    Big 172 (205)   Mid 205 (214)
//   TN  1536 x 2048 x 4096   Big 83 (85)     Mid 45 (41)    Small 52 (50)
struct MMCost {
  int bm, bn, threads, slots;
  double s1, s2, s3, full, part, dense;
};
constexpr MMCost kMMBigCost = {256, 256, 512, 256, 1.12, 1.64, 1.64, 9.0, 9.0, 14.0};
constexpr MMCost kMMMidCost = {128, 128, 256, 512, 0.62, 0.66, 0.96, 9.0, 4.0, 7.5};
constexpr MMCost kMMWideCost = {64, 128, 512, 512, 0.30, 0.36, 0.65, 6.5, 3.8, 2.3};
constexpr MMCost kMMSmallCost = {64, 64, 256, 512, 0.20, 0.23, 0.40, 5.0, 3.5, 1.7};
constexpr MMCost kMMLongCost = {128, 256, 256, 512, 1.00, 1.20, 1.90, 11.0, 5.0, 12.0};
constexpr MMCost kMMDeepCost = {128, 128, 512, 256, 0.41, 0.61, 0.61, 6.0, 4.0, 4.5};

// m tiles of row blocks: of `rows` rows in one block (E = 0), or spread over E
// experts, where about half a tile per expert in use is left over and none has
// less than one.
inline double mm_row_tiles(int bm, int rows, int E) {
  if (E == 0) return (rows + bm - 1) / bm;
  const double act = rows < E ? rows : E, n = static_cast<double>(rows) / bm + 0.5 * act;
  return n > act ? n : act;
}
// Most blocks of row-grouped tiles over all ways to cut the rows: a partial tile per
// expert (E 0: no experts).
inline long long mm_most_row_tiles(int bm, int rows, int E) {
  return rows / bm + (E == 0 ? 1LL : rows < E ? rows : E);
}
// Dense: `epi` us per 65536 results of a CU for activations.
inline double mm_cost(const MMCost& c, double tiles, double stages, bool dense = false,
                      double epi = 0.0) {
  const double full = __builtin_floor(tiles / c.slots), rem = tiles - full * c.slots;
  const double act = epi * c.bm * c.bn / 65536;
  double cost = full * (stages * c.s3 + (dense ? c.dense + act * c.slots / 256 : c.full));
  if (rem > 0) {
    // a CU with two blocks is done last, however few of them there are
    const double s = rem <= 64    ? c.s1
                     : rem <= 256 ? c.s1 + (c.s2 - c.s1) * (rem - 64) / 192
                     : dense      ? 0.87 * c.s3
                                  : c.s2 + (c.s3 - c.s2) * (rem - 256) / (c.slots - 256);
    cost += stages * s + c.part + act * (rem > 256 ? 2 : 1);
  }
  return cost;
}
// The cheapest geometry for row-grouped products (NT, NN): 0 Big, 1 Mid, 2 Wide,
// 3 Small, 4 Long, 5 Deep (dense only). Experts of few rows are bound by streaming their weights, which
// the low tiles keep most loads in flight for (128 experts x 1536 x 2048: 8192 rows
// Wide 181, Long 207, Mid 216, Big 249 us; 4096 rows 166, -, 189, 200).
struct MMPick {
  int geom;
  double cost;   // us
};
inline MMPick mm_pick_rows(int rows, int E, int ndim, int kdim, int act = 0) {
  // 8192 x 4096 x 1024: silu + 9 us in Big, gelu + 18; Mid + 7 and + 14 by this
  const double epi = E != 0 ? 0.0 : act == 3 ? 12.0 : act == 2 || act == kActSwiglu ? 6.0 : 0.0;
  const MMCost* const table[6] = {&kMMBigCost, &kMMMidCost, &kMMWideCost, &kMMSmallCost,
                                  &kMMLongCost, &kMMDeepCost};
  const bool low = E > 1 && rows <= 96LL * (rows < E ? rows : E);
  MMPick best = {0, 1e300};
  for (int i = 0; i < (E == 0 ? 6 : 5); ++i) {
    const MMCost& c = *table[i];
    if (low && c.bm > 64) continue;
    const int nt = (ndim + c.bn - 1) / c.bn;
    if (!mm_fits(mm_most_row_tiles(c.bm, rows, E) * nt, c.threads)) continue;
    const double cost = mm_cost(c, mm_row_tiles(c.bm, rows, E) * nt,
                                (kdim + 63) / 64, E == 0, epi);
    if (cost < best.cost) best = {i, cost};
  }
  return best;
}

// Results of more than the L2s' 32 MB go past them (see mm_put16), if their rows are
// whole cache lines: lines that two tiles write in part would be written twice
// (53 experts x 3552 x 232 bf16: 42 us with the hint, 21 without).
inline void mm_set_stream(MMArgs& a, long long rows, long long cols) {
  const long long row = cols * (a.c_f32 ? 4 : 2), z_row = a.z ? 2LL * a.ndim : 0;
  a.stream_out = rows * (row + z_row) > (32LL << 20) && row % 128 == 0 && z_row % 128 == 0;
}

// Fills in what the kernel needs of the geometry; returns the grid (a multiple of 8).
template <int MODE, class G>
long long mm_prepare(MMArgs& a) {
  long long tiles;
  const bool swiglu = MODE == kModeNT && a.act == kActSwiglu;
  a.nt = swiglu ? (a.ndim / 2 + G::BN / 2 - 1) / (G::BN / 2) : (a.ndim + G::BN - 1) / G::BN;
  if (MODE == kModeTN) {
    a.mt = (a.mdim + G::BM - 1) / G::BM;
    tiles = static_cast<long long>(a.E) * a.splits * a.mt * a.nt;
    a.xm = 0;
    if (a.E > 1) {
      // the split of 8 XCDs that pads least, then the one that reads least: a
      // slice reads its part of both operands
      long long best = -1;
      for (int xm = 1; xm <= 8; xm *= 2) {
        const long long tm = (a.mt + xm - 1) / xm, tn = (a.nt + 8 / xm - 1) / (8 / xm);
        const long long key = tm * tn * 1000000 + tm * G::BM + tn * G::BN;
        if (best < 0 || key < best) {
          best = key;
          a.xm = xm;
          tiles = 8 * tm * tn * a.E * a.splits;
        }
      }
    }
    mm_set_stream(a, static_cast<long long>(a.E) * a.splits * a.mdim, a.ndim);
  } else {
    mm_set_stream(a, static_cast<long long>(a.rows) * a.splits, swiglu ? a.ndim / 2 : a.ndim);
    tiles = mm_most_row_tiles(G::BM, a.rows, a.offsets ? a.E : 0) * a.nt * a.splits;
  }
  return (tiles + 7) / 8 * 8;
}

// Dynamic LDS of a kernel: the attribute is set once per device (threads that
// race set it twice).
struct MMReady {
  std::atomic<bool> device[moe_api::kMaxDevices];
  hipError_t set(const void* kernel, int lds) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 0 || dev >= moe_api::kMaxDevices) return hipErrorInvalidDevice;
    if (!device[dev].load(std::memory_order_acquire)) {
      e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
      device[dev].store(true, std::memory_order_release);
    }
    return hipSuccess;
  }
};

template <class T, int MODE, class G>
hipError_t mm_launch(MMArgs a, hipStream_t s, bool check) {
  const long long grid = mm_prepare<MODE, G>(a);
  if (grid == 0) return hipSuccess;
  if (!mm_fits(grid, G::kThreads)) return hipErrorInvalidConfiguration;
  if (check) return hipSuccess;
  static MMReady ready;
  const hipError_t e = ready.set(reinterpret_cast<const void*>(&mm_kernel<T, MODE, G>), G::kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((mm_kernel<T, MODE, G>), dim3(static_cast<unsigned>(grid)),
                     dim3(G::kThreads), G::kLds, s,
                     static_cast<const uint8_t*>(a.A), static_cast<const uint8_t*>(a.B), a);
  return hipGetLastError();
}

}  // namespace moe
