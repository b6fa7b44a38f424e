// Weight gradients (TN): dW = dz^T x over the rows of each expert.
#include "launch_block.h"
#include "mm_launch.h"

namespace moe {

using TNMid = MMGeom<128, 128, 2, 2, 64, 2, 2>;

// Parts an expert's rows are cut into: where the output tiles alone leave CUs
// idle, the contraction is split (each part a float32 product in the
// workspace, added in order), down to parts of four stages.
int mm_tn_splits(int rows, int E, int mdim, int ndim) {
  const long long tiles = static_cast<long long>(E) * ((mdim + TNMid::BM - 1) / TNMid::BM) *
                          ((ndim + TNMid::BN - 1) / TNMid::BN);
  const long long most = rows / E / (4 * TNMid::BK);
  long long s = 512 / tiles;
  if (s > most) s = most;
  if (s > 32) s = 32;
  return s < 1 ? 1 : static_cast<int>(s);
}

hipError_t launch_mm_tn(const MMArgs& a, bool fp16, hipStream_t s) {
  return fp16 ? mm_launch<fp16_tag, kModeTN, TNMid>(a, s) : mm_launch<bf16_tag, kModeTN, TNMid>(a, s);
}

}  // namespace moe
