// Sums of float32 parts over a column (a bias gradient's strips of rows).
#pragma once
#include "launch_block.h"
#include "mm.h"

namespace moe {

__device__ __forceinline__ void store_as(void* out, long long i, float v, int type) {
  if (type == 2) static_cast<float*>(out)[i] = v;
  else if (type == 0) static_cast<uint16_t*>(out)[i] = f32_to_bf16(v);
  else static_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(pack2<fp16_tag>(v, 0.0f));
}

// A block of 256 threads takes 32 columns, 8 runs of parts; the runs are joined in
// order.
inline unsigned sum_parts_blocks(const PartSum& a) {
  return a.out ? (static_cast<unsigned>(a.n) + 31) / 32 : 0;
}
__device__ __forceinline__ void sum_parts_block(const PartSum& a, uint32_t bid) {
  __shared__ float red[8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = static_cast<int>(bid) * 32 + tx;
  const int run = (a.parts + 7) / 8, p0 = ty * run, p1 = min(p0 + run, a.parts);
  float v = 0.0f;
  if (col < a.n)
#pragma unroll 8
    for (int p = p0; p < p1; ++p) v += a.part[static_cast<size_t>(p) * a.n + col];
  red[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && col < a.n) {
    for (int y = 1; y < 8; ++y) v += red[y][tx];
    store_as(a.out, col, v, a.out_type);
  }
}

}  // namespace moe
