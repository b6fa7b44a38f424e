// Weight gradients (TN): dW = dz^T x over the rows of each expert.
#include "launch_block.h"
#include "mm_grad.h"

namespace moe {
namespace {

template <class T>
hipError_t launch(const MMArgs& a, int geom, hipStream_t s, bool check) {
  switch (geom) {
    case 0: return mm_launch<T, kModeTN, MMBig>(a, s, check);
    case 1: return mm_launch<T, kModeTN, MMTall>(a, s, check);
    case 2: return mm_launch<T, kModeTN, MMMid>(a, s, check);
    default: return mm_launch<T, kModeTN, MMSmall>(a, s, check);
  }
}

}  // namespace

hipError_t launch_mm_tn(const MMArgs& a, int geom, bool fp16, hipStream_t s, bool check) {
  return fp16 ? launch<fp16_tag>(a, geom, s, check) : launch<bf16_tag>(a, geom, s, check);
}

}  // namespace moe
