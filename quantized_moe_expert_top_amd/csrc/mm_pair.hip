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
hipError_t launch(MMArgs nn, MMArgs tn, const PartSum& sum, hipStream_t s) {
  const long long tb = mm_prepare<kModeTN, G>(tn), nb = mm_prepare<kModeNN, G>(nn),
                  grid = tb + nb + sum_parts_blocks(sum);
  if (!mm_fits(grid, G::kThreads, (nn.rows / G::BM + 1LL) * nn.nt, nn.E))
    return hipErrorInvalidConfiguration;
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

// 1 Mid, 2 Small, 0 apart: where one launch is expected to beat two (3 us for the
// second launch and its start).
int mm_pair_pick(int rows, int E, int N, int K) {
  const bool grouped = E > 0;
  const TNPlan tn = mm_plan_tn(rows, grouped ? E : 1, N, K);
  const double apart = tn.cost + mm_pick_rows(rows, E, K, N).cost + 3.0;
  const int groups = grouped ? E : 1;
  double stages = static_cast<double>(rows) / groups / 64 + (grouped ? 0.5 : 0.0);
  if (stages < 1.0) stages = 1.0;
  int best = 0;
  double at = apart;
  const MMCost* const table[2] = {&kMMMidCost, &kMMSmallCost};
  for (int i = 0; i < 2; ++i) {
    const MMCost& c = *table[i];
    const double kt = (K + c.bn - 1) / c.bn;
    const double cost = pair_cost(c, groups * ((N + c.bm - 1) / c.bm) * kt, stages,
                                  mm_row_tiles(c.bm, rows, E) * kt, (N + 63) / 64);
    if (cost < at) {
      at = cost;
      best = i + 1;
    }
  }
  return best;
}

hipError_t launch_mm_pair(const MMArgs& nn, const MMArgs& tn, const PartSum& sum, int pick,
                          bool fp16, hipStream_t s) {
  if (pick == 1)
    return fp16 ? launch<fp16_tag, MMMid>(nn, tn, sum, s) : launch<bf16_tag, MMMid>(nn, tn, sum, s);
  return fp16 ? launch<fp16_tag, MMSmall>(nn, tn, sum, s) : launch<bf16_tag, MMSmall>(nn, tn, sum, s);
}

}  // namespace moe
