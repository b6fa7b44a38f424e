// Row gradients (NN): dx = dz W.
#include "launch_block.h"
#include "mm_launch.h"

namespace moe {
namespace {

template <class T>
hipError_t launch(const MMArgs& a, int geom, hipStream_t s) {
  switch (geom) {
    case 0: return mm_launch<T, kModeNN, MMBig>(a, s);
    case 1: return mm_launch<T, kModeNN, MMMid>(a, s);
    case 2: return mm_launch<T, kModeNN, MMWide>(a, s);
    case 3: return mm_launch<T, kModeNN, MMSmall>(a, s);
    case 4: return mm_launch<T, kModeNN, MMLong>(a, s);
    default: return mm_launch<T, kModeNN, MMDeep>(a, s);
  }
}

}  // namespace

hipError_t launch_mm_nn(const MMArgs& a, int geom, bool fp16, hipStream_t s) {
  return fp16 ? launch<fp16_tag>(a, geom, s) : launch<bf16_tag>(a, geom, s);
}

}  // namespace moe
