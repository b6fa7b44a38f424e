// Both gradients of a product in one launch: the weight gradient's tiles (TN, long
// contractions, often too few to fill the chip) first, the row gradient's (NN)
// behind them in the slots they leave. 4093 x 2048 x 1536 fp16: NN 31 us (one full
// round) and TN 43 us (192 of 512 slots) by themselves. The bias gradient's last sum
// goes along in the blocks after them, which start as the first tiles end (a launch
// of its own: 4.6 us).
#include "launch_block.h"
#include "mm_grad.h"
#include "part_sum.h"

namespace moe {
namespace {

template <class T, class G>
__global__ __launch_bounds__(G::kThreads, G::WPE) void mm_pair_kernel(
    const uint8_t* __restrict__ dz, const uint8_t* __restrict__ x, const uint8_t* __restrict__ w,
    const MMArgs tn, const MMArgs nn, const PartSum sum, uint32_t tn_blocks, uint32_t nn_blocks) {
  static_assert(G::kThreads == 256, "the sum's blocks");
  if (blockIdx.x < tn_blocks) mm_tile<T, kModeTN, G>(dz, x, tn, blockIdx.x);
  else if (blockIdx.x < tn_blocks + nn_blocks)
    mm_tile<T, kModeNN, G>(dz, w, nn, blockIdx.x - tn_blocks);
  else sum_parts_block(sum, blockIdx.x - tn_blocks - nn_blocks);
}

template <class T, class G>
hipError_t launch(MMArgs nn, MMArgs tn, const PartSum& sum, hipStream_t s, bool check) {
  const long long tb = mm_prepare<kModeTN, G>(tn), nb = mm_prepare<kModeNN, G>(nn),
                  grid = tb + nb + sum_parts_blocks(sum);
  if (!mm_fits(grid, G::kThreads)) return hipErrorInvalidConfiguration;
  if (check) return hipSuccess;
  static MMReady ready;
  const hipError_t e = ready.set(reinterpret_cast<const void*>(&mm_pair_kernel<T, G>), G::kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((mm_pair_kernel<T, G>), dim3(static_cast<unsigned>(grid)),
                     dim3(G::kThreads), G::kLds, s, static_cast<const uint8_t*>(tn.A),
                     static_cast<const uint8_t*>(tn.B), static_cast<const uint8_t*>(nn.B), tn, nn, sum,
                     static_cast<uint32_t>(tb), static_cast<uint32_t>(nb));
  return hipGetLastError();
}

// us of both in one launch of geometry c: all slots busy with the stages of both,
// and no less than the longer tile by itself
double pair_cost(const MMCost& c, double tn_tiles, double tn_stages, double nn_tiles,
                 double nn_stages) {
  const double tiles = tn_tiles + nn_tiles;
  const double work = tn_tiles * (tn_stages * c.s3 + c.full) + nn_tiles * (nn_stages * c.s3 + c.full);
  const double longest = tn_stages > nn_stages ? tn_stages : nn_stages;
  const double alone = mm_cost(c, tiles < c.slots ? tiles : c.slots, longest);
  return work / c.slots > alone ? work / c.slots : alone;
}

}  // namespace

// The cheapest way: apart, with 3 us for the second launch and its start, or in one
// launch; contractions cut where that fills the chip (only without experts in the
// row gradient; with experts only apart).
static MMBackwardPlan plan_of(int rows, int E, int N, int K) {
  const bool grouped = E > 0;
  const int groups = grouped ? E : 1;
  const MMPick nn1 = mm_pick_rows(rows, E, K, N);
  MMPlan nn[2] = {{nn1.geom, 1, nn1.cost}, {0, 1, 1e300}};
  if (!grouped) nn[1] = mm_plan_nn_split(rows, K, N);
  const MMPlan tn[2] = {mm_plan_tn(rows, groups, N, K, false), mm_plan_tn(rows, groups, N, K, true)};
  MMBackwardPlan best = {0, nn[0].geom, 1, tn[0].geom, 1};
  double at = 1e300;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) {
      const double cost = nn[i].cost + tn[j].cost + 3.0 + (i || j ? kMMSplitLaunch : 0.0);
      if (cost < at) {
        at = cost;
        best = {0, nn[i].geom, nn[i].splits, tn[j].geom, tn[j].splits};
      }
    }
  const double tn_stages = mm_tn_stages(rows, groups), nn_stages = (N + 63) / 64;
  const int most_dx = grouped ? 1 : mm_most_dx_splits(rows, N, K),
            most_dw = grouped ? 1 : mm_most_dw_splits(rows, 1, N, K);
  const MMCost* const table[2] = {&kMMMidCost, &kMMSmallCost};
  for (int i = 0; i < 2; ++i) {
    const MMCost& c = *table[i];
    const double kt = (K + c.bn - 1) / c.bn;
    const double tn_tiles = groups * static_cast<double>((N + c.bm - 1) / c.bm) * kt,
                 nn_tiles = mm_row_tiles(c.bm, rows, E) * kt;
    if (!mm_fits(static_cast<long long>(tn_tiles) * most_dw +
                     mm_most_row_tiles(c.bm, rows, E) * static_cast<long long>(kt) * most_dx +
                     (N + 31) / 32 + 16, c.threads))
      continue;
    for (int a = 1; a <= most_dx; a *= 2)
      for (int b = 1; b <= most_dw; b *= 2) {
        const double cost = pair_cost(c, tn_tiles * b, tn_stages / b, nn_tiles * a, nn_stages / a) +
                            mm_split_cost(static_cast<double>(rows) * K, a) +
                            mm_split_cost(static_cast<double>(N) * K, b) +
                            (a > 1 || b > 1 ? kMMSplitLaunch : 0.0);
        if (cost < at) {
          at = cost;
          best = {i + 1, i == 0 ? 1 : 3, a, i == 0 ? 2 : 3, b};
        }
      }
  }
  return best;
}

MMBackwardPlan mm_backward_plan(int rows, int E, int N, int K) {
  // this thread's last plans: one takes some hundred evaluations, about as long as
  // a launch
  struct Kept {
    bool set;
    int rows, E, N, K;
    MMBackwardPlan plan;
  };
  static thread_local Kept kept[16];
  const uint32_t h = (static_cast<uint32_t>(rows) * 2654435761u) ^ (static_cast<uint32_t>(N) * 40503u) ^
                     (static_cast<uint32_t>(K) * 9973u) ^ (static_cast<uint32_t>(E) * 31u);
  Kept& k = kept[(h ^ (h >> 15)) & 15];
  if (!k.set || k.rows != rows || k.E != E || k.N != N || k.K != K)
    k = {true, rows, E, N, K, plan_of(rows, E, N, K)};
  return k.plan;
}

size_t mm_backward_parts(int rows, int E, int N, int K) {
  const int groups = E > 0 ? E : 1, dw = mm_most_dw_splits(rows, groups, N, K);
  size_t n = dw > 1 ? (static_cast<size_t>(groups) * dw * N * K * 4 + 255) & ~size_t{255} : 0;
  if (E == 0) {
    // for every count of rows up to this one
    const size_t most = mm_most_splits((N + 63) / 64, 1), all = most * rows * K * 4,
                 cap = static_cast<size_t>(kMMSplitTiles) * 64 * 64 * 4;
    if (most > 1) n += ((all < cap ? all : cap) + 255) & ~size_t{255};
  }
  return n;
}

hipError_t launch_mm_pair(const MMArgs& nn, const MMArgs& tn, const PartSum& sum, int pair,
                          bool fp16, hipStream_t s, bool check) {
  if (pair == 1)
    return fp16 ? launch<fp16_tag, MMMid>(nn, tn, sum, s, check)
                : launch<bf16_tag, MMMid>(nn, tn, sum, s, check);
  return fp16 ? launch<fp16_tag, MMSmall>(nn, tn, sum, s, check)
              : launch<bf16_tag, MMSmall>(nn, tn, sum, s, check);
}

}  // namespace moe
