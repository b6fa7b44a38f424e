// Row gradients (NN): dx = dz W.
#include "launch_block.h"
#include "mm_launch.h"

namespace moe {

using NNMid = MMGeom<128, 128, 2, 2, 64, 2, 2>;

hipError_t launch_mm_nn(const MMArgs& a, bool fp16, hipStream_t s) {
  return fp16 ? mm_launch<fp16_tag, kModeNN, NNMid>(a, s) : mm_launch<bf16_tag, kModeNN, NNMid>(a, s);
}

}  // namespace moe
