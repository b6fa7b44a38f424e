// Forward products (NT): z = x W^T with bias, activation and residual.
#include "launch_block.h"
#include "mm_few.h"
#include "mm_launch.h"

namespace moe {
namespace {

template <class T>
hipError_t launch(const MMArgs& a, hipStream_t s) {
  const int E = a.offsets ? a.E : 0;
  // Few rows, or few results of a long K: the kernel that splits K over a block's
  // waves. Measured at 2 x 4096 x 7168: 11.7 us against 23.2 (Small); 32 rows: 22.3
  // against 23.5. Where several experts are in use the tiles mostly fill the chip by
  // themselves.
  const MMPick pick = mm_pick_rows(a.rows, E, a.ndim, a.kdim, a.act);
  const double f1 = mm_few_cost(1, a.rows, E, a.ndim, a.kdim),
               f2 = E == 0 ? mm_few_cost(2, a.rows, E, a.ndim, a.kdim) : 1e300;
  if ((E == 0 && a.rows <= 16) || f1 < pick.cost || f2 < pick.cost)
    return a.rows <= 16 || f1 <= f2 ? mm_few_launch<T, 1, 8, 2>(a, s)
                                    : mm_few_launch<T, 2, 8, 2>(a, s);
  switch (pick.geom) {
    case 0: return mm_launch<T, kModeNT, MMBig>(a, s);
    case 1: return mm_launch<T, kModeNT, MMMid>(a, s);
    case 2: return mm_launch<T, kModeNT, MMWide>(a, s);
    case 3: return mm_launch<T, kModeNT, MMSmall>(a, s);
    case 4: return mm_launch<T, kModeNT, MMLong>(a, s);
    default: return mm_launch<T, kModeNT, MMDeep>(a, s);
  }
}

}  // namespace

hipError_t launch_mm_nt(const MMArgs& a, bool fp16, hipStream_t s) {
  return fp16 ? launch<fp16_tag>(a, s) : launch<bf16_tag>(a, s);
}

}  // namespace moe
