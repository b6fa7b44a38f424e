// Token rows to int8 codes with a scale per row (moe_quant_rows), bound by the bytes of
// the rows: each is read once and stays in registers between its maximum and its codes. 8192 x 7168:
// 30 us, 176 MB at 5.9 TB/s; 61 x 2048 3 us, the launch.
#include "launch_int8.h"
#include "quant.h"

namespace moe {
namespace {

// T: the 16-bit type, or any where F32. A row is held by WPR waves, NC chunks of 8 per
// thread; WPR = 1 puts four rows in a block.
template <class T, bool F32, int WPR, int NC>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void quant_rows_kernel(
    const void* __restrict__ x, int rows, int K, int8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int kRows = WPR == 1 ? 4 : 1, kRowThreads = WPR * kWave;
  __shared__ uint32_t red[WPR];
  const int rt = WPR == 1 ? (threadIdx.x & (kWave - 1)) : threadIdx.x;
  const int t = blockIdx.x * kRows + (WPR == 1 ? threadIdx.x >> 6 : 0);
  if (t >= rows) return;   // whole waves; with WPR > 1, whole blocks
  const int C = K / 8;
  const size_t row = static_cast<size_t>(t) * K;
  Row8<T, F32> v[NC];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) v[i].load(x, row + min(rt + i * kRowThreads, C - 1) * 8);   // past the row: its last
#pragma unroll
  for (int i = 0; i < NC; ++i) m = amax8(v[i], m);
  m = wave_max_u32(m);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) m = max_u32(m, red[w]);
  }
  const RowScale s = row_scale(m);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = rt + i * kRowThreads;
    if (c >= C) continue;
    float f[8];
    v[i].values(f);
    *reinterpret_cast<uint2*>(q + row + c * 8) = codes8(f, s);
  }
  if (rt == 0) scale[t] = s.s;
}

template <class T, bool F32>
hipError_t launch(const void* x, int rows, int K, int8_t* q, float* scale, hipStream_t s) {
  const int C = K / 8;
  if (C <= 256) {
    const unsigned four = (static_cast<unsigned>(rows) + 3) / 4;
    if (C <= 64) quant_rows_kernel<T, F32, 1, 1><<<four, 256, 0, s>>>(x, rows, K, q, scale);
    else if (C <= 128) quant_rows_kernel<T, F32, 1, 2><<<four, 256, 0, s>>>(x, rows, K, q, scale);
    else quant_rows_kernel<T, F32, 1, 4><<<four, 256, 0, s>>>(x, rows, K, q, scale);
  } else if (C <= 512) {
    quant_rows_kernel<T, F32, 4, 2><<<rows, 256, 0, s>>>(x, rows, K, q, scale);
  } else if (C <= 1024) {
    quant_rows_kernel<T, F32, 4, 4><<<rows, 256, 0, s>>>(x, rows, K, q, scale);
  } else {
    quant_rows_kernel<T, F32, 16, 8><<<rows, 1024, 0, s>>>(x, rows, K, q, scale);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_rows(const void* x, int x_type, int rows, int K, int8_t* q, float* scale,
                             hipStream_t s) {
  // one launch holds less than 2^32 threads: 2^21 rows of 1024
  constexpr int kLaunchRows = 1 << 21;
  const size_t size = x_type == 2 ? 4 : 2;
  for (int t0 = 0; t0 < rows;) {
    const int n = rows - t0 < kLaunchRows ? rows - t0 : kLaunchRows;
    const size_t at = static_cast<size_t>(t0) * K;
    const void* from = static_cast<const uint8_t*>(x) + at * size;
    const hipError_t e = x_type == 2   ? launch<bf16_tag, true>(from, n, K, q + at, scale + t0, s)
                         : x_type == 1 ? launch<fp16_tag, false>(from, n, K, q + at, scale + t0, s)
                                       : launch<bf16_tag, false>(from, n, K, q + at, scale + t0, s);
    if (e != hipSuccess) return e;
    t0 += n;
    if (n < kLaunchRows) break;
  }
  return hipSuccess;
}

}  // namespace moe
