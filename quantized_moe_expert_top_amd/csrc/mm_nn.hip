// Row gradients (NN): dx = dz W.
#include "launch_block.h"
#include "mm_launch.h"

namespace moe {
namespace {

template <class T>
hipError_t launch(const MMArgs& a, int geom, hipStream_t s, bool check) {
  switch (geom) {
    case 0: return mm_launch<T, kModeNN, MMBig>(a, s, check);
    case 1: return mm_launch<T, kModeNN, MMMid>(a, s, check);
    case 2: return mm_launch<T, kModeNN, MMWide>(a, s, check);
    case 3: return mm_launch<T, kModeNN, MMSmall>(a, s, check);
    case 4: return mm_launch<T, kModeNN, MMLong>(a, s, check);
    default: return mm_launch<T, kModeNN, MMDeep>(a, s, check);
  }
}

}  // namespace

hipError_t launch_mm_nn(const MMArgs& a, int geom, bool fp16, hipStream_t s, bool check) {
  return fp16 ? launch<fp16_tag>(a, geom, s, check) : launch<bf16_tag>(a, geom, s, check);
}

}  // namespace moe
