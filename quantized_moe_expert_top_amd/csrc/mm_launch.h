// Host side of the tile products: launch of one geometry, grid sizes.
#pragma once
#include "mm.h"

namespace moe {

template <class T, int MODE, class G>
hipError_t mm_launch(MMArgs a, hipStream_t s) {
  long long tiles;
  const bool swiglu = MODE == kModeNT && a.act == kActSwiglu;
  a.nt = swiglu ? (a.ndim / 2 + G::BN / 2 - 1) / (G::BN / 2) : (a.ndim + G::BN - 1) / G::BN;
  if (MODE == kModeTN) {
    a.mt = (a.mdim + G::BM - 1) / G::BM;
    tiles = static_cast<long long>(a.E) * a.splits * a.mt * a.nt;
  } else {
    // an upper bound over all ways to cut the rows: a partial tile per expert
    const long long partial = a.offsets ? (a.rows < a.E ? a.rows : a.E) : 1;
    tiles = (a.rows / G::BM + partial) * a.nt;
  }
  const long long grid = (tiles + 7) / 8 * 8;
  if (grid == 0) return hipSuccess;
  if (grid >= (1LL << 31)) return hipErrorInvalidConfiguration;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&mm_kernel<T, MODE, G>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, G::kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((mm_kernel<T, MODE, G>), dim3(static_cast<unsigned>(grid)),
                     dim3(G::kThreads), G::kLds, s, a);
  return hipGetLastError();
}

}  // namespace moe
