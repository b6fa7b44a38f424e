// Forward products (NT): z = x W^T with bias, activation and residual.
#include "launch_block.h"
#include "mm_launch.h"

namespace moe {

using NTMid = MMGeom<128, 128, 2, 2, 64, 2, 2>;

hipError_t launch_mm_nt(const MMArgs& a, bool fp16, hipStream_t s) {
  return fp16 ? mm_launch<fp16_tag, kModeNT, NTMid>(a, s) : mm_launch<bf16_tag, kModeNT, NTMid>(a, s);
}

}  // namespace moe
