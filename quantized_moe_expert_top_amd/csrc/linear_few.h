// Dense int8 products of up to 16 rows (moe_linear_w8a8): y = act(z) + residual.
//
// A block takes tiles of 16 weight rows (SwiGLU: 8 gate rows and the 8 matching up rows),
// one after another, and its waves split K: wave w takes the 128-byte steps w, w + 8, ... of
// each through its ring (few.h), without a stop between tiles. The waves' integer sums are
// added in LDS, exactly, so that no result depends on timing. 2 x 7168 -> SwiGLU 4096: 29.4 MB
// in 9.0 us with its launch (20480 columns: 147 MB in 24, 6.1 TB/s).
#pragma once
#include "few.h"
#include "launch_int8.h"
#include "norm_rows.h"

namespace moe {

constexpr int kLinearTiles = 8;   // most tiles of a block

// VALUES: x holds values of XT, whose codes the block makes; otherwise codes and scales.
// O: the 16-bit type of y, or any with OUT32.
template <bool VALUES, class XT, class O, bool OUT32, int D>
__global__ __launch_bounds__(kFewThreads, 2) void linear_few_kernel(const LinearI8 a, const void* x) {
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];   // ring, codes
  __shared__ int s_acc[kLinearTiles][16][17];
  __shared__ float s_scale[kFewTokens];
  __shared__ uint32_t s_amax[kFewTokens];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, kg = lane >> 4;
  const int K = a.K, M = a.rows, stride = K + 16;
  const bool swiglu = a.act == kActSwiglu;   // uniform
  const int half = a.N / 2, width = swiglu ? half : a.N, cols = swiglu ? 8 : 16;
  uint8_t* ring = few_lds + wv * (D * kFewSlot);
  uint8_t* codes = few_lds + kFewWaves * D * kFewSlot;

  // rows of x first: loads return in order, so that these are not waited for behind the
  // ring's
  FewRows<XT, false> made;
  FewCodes copied;
  if constexpr (VALUES) {
    made.get(x, M, K);
    if (tid < M) s_amax[tid] = 0;
  } else {
    copied.get(a.q, a.q_scale, M, K);
  }
  for (int i = tid; i < kLinearTiles * 16 * 17; i += kFewThreads) (&s_acc[0][0][0])[i] = 0;
  // the first output of this thread: what is added to it is asked for here
  const int tiles = (width + cols - 1) / cols, b = blockIdx.x;
  const int mine = (tiles - b + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  struct Added {
    float s, s_up, bias, bias_up;
    uint32_t res;   // as it is stored
  };
  auto place = [&](int i, int& t, int& r, int& c, int& col) {   // output i of the block
    t = i / (M * cols);
    r = (i - t * M * cols) / cols;
    c = i % cols;
    col = (b + t * static_cast<int>(gridDim.x)) * cols + c;
    return t < mine && col < width;
  };
  auto added = [&](int i) {
    Added v = {0.0f, 0.0f, 0.0f, 0.0f, 0};
    int t, r, c, col;
    if (!place(i, t, r, c, col)) return v;
    v.s = a.w_scale[col];
    if (swiglu) v.s_up = a.w_scale[half + col];
    if (a.bias) {
      v.bias = a.bias[col];
      if (swiglu) v.bias_up = a.bias[half + col];
    }
    if (a.residual) {
      const size_t at = static_cast<size_t>(r) * width + col;
      if (OUT32) v.res = static_cast<const uint32_t*>(a.residual)[at];
      else v.res = static_cast<const uint16_t*>(a.residual)[at];
    }
    return v;
  };
  const Added first = added(tid);
  const int steps = (K + kFewStep - 1) / kFewStep;
  const int each = (steps - wv + kFewWaves - 1) / kFewWaves;   // steps of this wave a tile
  const int total = mine * each;
  const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(a.w, static_cast<uint32_t>(a.N) * K);
  const int lrow = lane >> 3, chunk = few_chunk(lane);
  int it = 0, is = 0;   // issue cursor: tile, step
  uint32_t off0 = 0, off1 = 0;
  auto enter = [&](int t) {
    const int n0 = (b + t * static_cast<int>(gridDim.x)) * cols;
    // SwiGLU: ring rows 4 q + {0, 1} are gate rows 2 q + {0, 1}, 4 q + {2, 3} the matching up rows
    const int r0 = swiglu ? n0 + (lrow >> 2) * 2 + (lrow & 1) : n0 + lrow;
    const int r1 = swiglu ? r0 + 4 : r0 + 8;
    const int up = swiglu && (lrow & 2) ? half : 0;
    off0 = r0 < width ? __umul24(r0 + up, K) + chunk * 16 : kMMPastEnd;
    off1 = r1 < width ? __umul24(r1 + up, K) + chunk * 16 : kMMPastEnd;
  };
  auto issue = [&](int slot) {
    const int k0 = (wv + is * kFewWaves) * kFewStep;
    const bool in = it < mine && k0 + chunk * 16 < K;
    few_issue(ring + slot * kFewSlot, rs, off0 == kMMPastEnd ? off0 : off0 + k0, rs,
              off1 == kMMPastEnd ? off1 : off1 + k0, in);
    if (++is == each) {
      is = 0;
      if (++it < mine) enter(it);
    }
  };
  // not the whole ring before the codes are made: loads waiting to be issued would hold that
  // up. Issued by every wave, whether it has steps or not: the compiler counts them.
  constexpr int kFirst = VALUES ? D / 4 * 3 : D;
  if (total > 0) enter(0);
#pragma unroll
  for (int d = 0; d < kFirst; ++d) issue(d);
  if constexpr (VALUES) {
    few_barrier();   // s_amax is cleared
    made.amax(M, K, s_amax);
    few_barrier();
    made.put(M, K, s_amax, codes, stride, s_scale);
#pragma unroll
    for (int d = kFirst; d < D; ++d) issue(d);
  } else {
    copied.put(a.q, M, K, codes, stride, s_scale);
  }
  few_barrier();

  const uint8_t* xrow = codes + min(l16, M - 1) * stride;
  i32x4_t acc = {0, 0, 0, 0};
  for (int i = 0, slot = 0, t = 0, st = 0; i < total; ++i) {
    few_wait<D - 1>();
    i32x4_t w0, w1;
    few_read(ring + slot * kFewSlot, w0, w1);
    // past k the weights are zeros, and any codes will do
    const int k0 = (wv + st * kFewWaves) * kFewStep + kg * 16;
    const i32x4_t x0 = *reinterpret_cast<const i32x4_t*>(xrow + min(k0, K - 16));
    const i32x4_t x1 = *reinterpret_cast<const i32x4_t*>(xrow + min(k0 + 64, K - 16));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read
    issue(slot);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, x0, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, x1, acc, 0, 0, 0);
    slot = slot + 1 == D ? 0 : slot + 1;
    if (++st == each) {
      // lane: row l16 of x, weight rows 4 kg + [0, 4)
      few_settle(acc);
      if (l16 < M)
#pragma unroll
        for (int q = 0; q < 4; ++q) few_add(&s_acc[t][l16][kg * 4 + q], acc[q]);
      acc = i32x4_t{0, 0, 0, 0};
      st = 0;
      ++t;
    }
  }
  // no load to LDS outlives the block
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  few_barrier();
  for (int i = tid; i < mine * M * cols; i += kFewThreads) {
    int t, r, c, col;
    if (!place(i, t, r, c, col)) continue;
    const Added v = i == tid ? first : added(i);
    const float xs = s_scale[r];
    const int at = swiglu ? (c >> 1) * 4 + (c & 1) : c;
    float z = __builtin_fmaf(static_cast<float>(s_acc[t][r][at]) * xs, v.s, v.bias);
    if (swiglu) {
      const float up = __builtin_fmaf(static_cast<float>(s_acc[t][r][at + 2]) * xs, v.s_up, v.bias_up);
      z = silu_f32<OUT32>(z) * up;
    } else {
      z = act_f32<OUT32>(z, a.act);
    }
    if (a.residual) {
      float res = __uint_as_float(v.res), hi;
      if (!OUT32) unpack2<O>(v.res, res, hi);
      z += res;
    }
    const size_t to = static_cast<size_t>(r) * width + col;
    if (OUT32) static_cast<float*>(a.y)[to] = z;
    else static_cast<uint16_t*>(a.y)[to] = static_cast<uint16_t>(pack2<O>(z, 0.0f));
  }
}

}  // namespace moe
