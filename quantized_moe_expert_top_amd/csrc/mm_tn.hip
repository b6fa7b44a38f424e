// Weight gradients (TN): dW = dz^T x over the rows of each expert.
#include "launch_block.h"
#include "mm_grad.h"

namespace moe {
namespace {

template <class T>
hipError_t launch(const MMArgs& a, int geom, hipStream_t s) {
  switch (geom) {
    case 0: return mm_launch<T, kModeTN, MMBig>(a, s);
    case 1: return mm_launch<T, kModeTN, MMTall>(a, s);
    case 2: return mm_launch<T, kModeTN, MMMid>(a, s);
    default: return mm_launch<T, kModeTN, MMSmall>(a, s);
  }
}

}  // namespace

hipError_t launch_mm_tn(const MMArgs& a, int geom, bool fp16, hipStream_t s) {
  return fp16 ? launch<fp16_tag>(a, geom, s) : launch<bf16_tag>(a, geom, s);
}

}  // namespace moe
