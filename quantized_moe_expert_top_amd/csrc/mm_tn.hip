// Weight gradients (TN): dW = dz^T x over the rows of each expert.
#include "launch_block.h"
#include "mm_grad.h"

namespace moe {
namespace {

template <class T>
hipError_t launch(const MMArgs& a, hipStream_t s) {
  switch (mm_plan_tn(a.rows, a.E, a.mdim, a.ndim).geom) {
    case 0: return mm_launch<T, kModeTN, MMBig>(a, s);
    case 1: return mm_launch<T, kModeTN, MMTall>(a, s);
    case 2: return mm_launch<T, kModeTN, MMMid>(a, s);
    default: return mm_launch<T, kModeTN, MMSmall>(a, s);
  }
}

}  // namespace

int mm_tn_splits(int rows, int E, int mdim, int ndim) { return mm_plan_tn(rows, E, mdim, ndim).splits; }

hipError_t launch_mm_tn(const MMArgs& a, bool fp16, hipStream_t s) {
  return fp16 ? launch<fp16_tag>(a, s) : launch<bf16_tag>(a, s);
}

}  // namespace moe
