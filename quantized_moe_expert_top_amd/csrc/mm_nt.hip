// Forward products (NT): z = x W^T with bias, activation and residual.
#include "launch_block.h"
#include "mm_few.h"
#include "mm_launch.h"

namespace moe {
namespace {

template <class T>
hipError_t launch(const MMArgs& a, int plan, hipStream_t s, bool check) {
  switch (plan) {
    case 0: return mm_launch<T, kModeNT, MMBig>(a, s, check);
    case 1: return mm_launch<T, kModeNT, MMMid>(a, s, check);
    case 2: return mm_launch<T, kModeNT, MMWide>(a, s, check);
    case 3: return mm_launch<T, kModeNT, MMSmall>(a, s, check);
    case 4: return mm_launch<T, kModeNT, MMLong>(a, s, check);
    case 5: return mm_launch<T, kModeNT, MMDeep>(a, s, check);
    case 6: return mm_few_launch<T, 1, 8, 2>(a, s, check);
    default: return mm_few_launch<T, 2, 8, 2>(a, s, check);
  }
}

}  // namespace

int mm_forward_plan(int rows, int E, int N, int K, int act) {
  // Few rows, or few results of a long K: the kernel that splits K over a block's
  // waves. Measured at 2 x 4096 x 7168: 11.7 us against 23.2 (Small); 32 rows: 22.3
  // against 23.5. Where several experts are in use the tiles mostly fill the chip by
  // themselves.
  const MMPick pick = mm_pick_rows(rows, E, N, K, act);
  const double f1 = mm_few_cost(1, rows, E, N, K),
               f2 = E == 0 ? mm_few_cost(2, rows, E, N, K) : 1e300;
  if ((E == 0 && rows <= 16) || f1 < pick.cost || f2 < pick.cost)
    return rows <= 16 || f1 <= f2 ? 6 : 7;
  return pick.geom;
}

hipError_t launch_mm_nt(const MMArgs& a, int plan, bool fp16, hipStream_t s, bool check) {
  return fp16 ? launch<fp16_tag>(a, plan, s, check) : launch<bf16_tag>(a, plan, s, check);
}

}  // namespace moe
