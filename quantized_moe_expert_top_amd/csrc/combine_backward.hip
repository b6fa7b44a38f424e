// Gradients of the weighted combine and of the softmax over a token's picks.
//
//   dy[pos(t, j)] = w_tj dout_t        dw_tj = <dout_t, y[pos(t, j)]>
//   dlogits[t, id_tj] = w_tj (dw_tj - sum_i w_ti dw_ti),  0 elsewhere
//
// Bound by the bytes of y and dy. A block takes a token, a wave (16 lanes where
// rows are short) one pick at a time over the whole row, so a pick's dot product is
// one sum in a fixed order and the rows are in flight at once; dout comes from the
// caches after its first read.
#include "launch_block.h"
#include "mm.h"

namespace moe {
namespace {

constexpr int kMaxPicks = 32;

// DY: 0 bf16, 1 fp16, 2 float32. STREAM: past the caches (see mm_put16), where dy
// takes more than the L2s' 32 MB.
template <bool STREAM>
__device__ __forceinline__ void put16(i32x4_t w, void* p) {
  if constexpr (STREAM) __builtin_nontemporal_store(w, static_cast<i32x4_t*>(p));
  else *static_cast<i32x4_t*>(p) = w;
}
template <int DY, bool STREAM>
__device__ __forceinline__ void store_dy(void* dy, size_t at, const float (&v)[8]) {
  if constexpr (DY == 2) {
    float* q = static_cast<float*>(dy) + at;
    put16<STREAM>(__builtin_bit_cast(i32x4_t, f32x4_t{v[0], v[1], v[2], v[3]}), q);
    put16<STREAM>(__builtin_bit_cast(i32x4_t, f32x4_t{v[4], v[5], v[6], v[7]}), q + 4);
  } else {
    using T = typename std::conditional<DY == 0, bf16_tag, fp16_tag>::type;
    put16<STREAM>(mm_pack8<T>(v), static_cast<uint16_t*>(dy) + at);
  }
}

// Sum over LPG neighbouring lanes, in a fixed order; each gets it.
template <int LPG>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LPG == kWave) return wave_sum_f32(v);
#pragma unroll
  for (int d = LPG / 2; d > 0; d /= 2) v += __shfl_xor(v, d, kWave);
  return v;
}

// LPG lanes per pick: 16 for rows of up to 256 values, else a wave.
template <int DY, bool STREAM, int LPG>
__global__ __launch_bounds__(512) void combine_backward_kernel(
    const float* __restrict__ dout, const float* __restrict__ y, const int* __restrict__ slot_pos,
    const int* __restrict__ ids, const float* __restrict__ w, long long R, int H, int E, int k,
    void* __restrict__ dy, float* __restrict__ dw, float* __restrict__ dlogits) {
  __shared__ float sdw[kMaxPicks];
  __shared__ float swt[kMaxPicks];
  __shared__ int sid[kMaxPicks];
  const int t = blockIdx.x, lane = threadIdx.x % LPG, grp = threadIdx.x / LPG;
  const int groups = blockDim.x / LPG;
  const int C = H / 8;
  const float* drow = dout + static_cast<size_t>(t) * H;
  const bool need_dot = dw != nullptr || dlogits != nullptr;
  for (int j = grp; j < k; j += groups) {
    const size_t f = static_cast<size_t>(t) * k + j;
    long long p = slot_pos[f];
    p = p < 0 ? 0 : p >= R ? R - 1 : p;
    const float wj = w[f];
    const size_t row = static_cast<size_t>(p) * H;
    float dot = 0.0f;
#pragma unroll 4
    for (int c = lane; c < C; c += LPG) {
      const float4* d4 = reinterpret_cast<const float4*>(drow + c * 8);
      const float4 d0 = d4[0], d1 = d4[1];
      if (need_dot) {
        const float4* y4 = reinterpret_cast<const float4*>(y + row + c * 8);
        const float4 y0 = y4[0], y1 = y4[1];
        dot += d0.x * y0.x + d0.y * y0.y + d0.z * y0.z + d0.w * y0.w + d1.x * y1.x + d1.y * y1.y +
               d1.z * y1.z + d1.w * y1.w;
      }
      if (dy) {
        const float v[8] = {wj * d0.x, wj * d0.y, wj * d0.z, wj * d0.w,
                            wj * d1.x, wj * d1.y, wj * d1.z, wj * d1.w};
        store_dy<DY, STREAM>(dy, row + c * 8, v);
      }
    }
    if (need_dot) {
      dot = lanes_sum<LPG>(dot);
      if (lane == 0) {
        if (dw) dw[f] = dot;
        sdw[j] = dot;
        swt[j] = wj;
        if (dlogits) sid[j] = ids[f];
      }
    }
  }
  if (dlogits == nullptr) return;   // uniform
  __syncthreads();
  float mean = 0.0f;
  for (int j = 0; j < k; ++j) mean += swt[j] * sdw[j];
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float v = 0.0f;
    for (int j = 0; j < k; ++j) v += sid[j] == e ? swt[j] * (sdw[j] - mean) : 0.0f;
    dlogits[static_cast<size_t>(t) * E + e] = v;
  }
}

}  // namespace

hipError_t launch_combine_backward(const float* dout, const float* y, const int* slot_pos,
                                   const int* ids, const float* w, int T, int H, int E, int k,
                                   void* dy, int dy_type, float* dw, float* dlogits,
                                   hipStream_t s) {
  if (T == 0) return hipSuccess;
  // 5351 tokens x 9 picks x 120: 28 us with a wave per pick, 12 with 16 lanes
  const int lpg = H <= 256 ? 16 : kWave, most = 512 / lpg;
  const int passes = (k + most - 1) / most, groups = (k + passes - 1) / passes;
  const int threads = (groups * lpg + kWave - 1) / kWave * kWave;
  const long long R = static_cast<long long>(T) * k;
  const bool stream = dy && R * H * (dy_type == 2 ? 4 : 2) > (32LL << 20) &&
                      H % 64 == 0;   // rows of whole cache lines
  auto launch = [&](auto dyc, auto lpgc) {
    constexpr int DY = decltype(dyc)::value, LPG = decltype(lpgc)::value;
    // one launch holds less than 2^32 threads: 2^22 tokens of 512
    constexpr int kLaunchTokens = 1 << 22;
    for (long long t0 = 0; t0 < T; t0 += kLaunchTokens) {
      const unsigned n = static_cast<unsigned>(T - t0 < kLaunchTokens ? T - t0 : kLaunchTokens);
      const auto run = stream ? &combine_backward_kernel<DY, true, LPG>
                              : &combine_backward_kernel<DY, false, LPG>;
      run<<<n, threads, 0, s>>>(dout + t0 * H, y, slot_pos + t0 * k, ids ? ids + t0 * k : nullptr,
                                w + t0 * k, R, H, E, k, dy, dw ? dw + t0 * k : nullptr,
                                dlogits ? dlogits + t0 * E : nullptr);
    }
  };
  auto typed = [&](auto lpgc) {
    if (dy_type == 0) launch(std::integral_constant<int, 0>{}, lpgc);
    else if (dy_type == 1) launch(std::integral_constant<int, 1>{}, lpgc);
    else launch(std::integral_constant<int, 2>{}, lpgc);
  };
  if (lpg == 16) typed(std::integral_constant<int, 16>{});
  else typed(std::integral_constant<int, 64>{});
  return hipGetLastError();
}

}  // namespace moe
