// Forward products of few rows (decode): C = act(x W^T + bias) + residual with at
// most 16 MT rows per block, bound by the bytes of W.
//
// A block takes 16 rows of W (SwiGLU: 8 gate rows and the matching 8 up rows) and
// its waves split K among them: wave w takes the 64-k steps w, w + WAVES, ..., so
// the block reads 128 WAVES contiguous bytes of each row per round. Operands go
// from memory straight into the registers of v_mfma_f32_16x16x32 (each W value is
// used once: staging it would only add latency), U steps ahead. The waves'
// partial tiles are added in LDS in wave order, so the result does not depend
// on timing.
#pragma once
#include "mm_launch.h"

namespace moe {

template <class T>
__device__ __forceinline__ f32x4_t mfma16x16(frag_t a, frag_t b, f32x4_t c) {
  if constexpr (__is_same(T, bf16_tag))
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

template <class T, int MT, int WAVES, int U>
__global__ __launch_bounds__(WAVES * 64) void mm_few_kernel(const uint8_t* __restrict__ Ab,
                                                            const uint8_t* __restrict__ Bb,
                                                            const MMArgs a) {
  constexpr int BM = 16 * MT, NTHR = WAVES * kWave;
  __shared__ __attribute__((aligned(16))) float part[WAVES][BM][16];
  __shared__ int sm_tile[NTHR / kWave + 4];
  MMTile t;
  if (!mm_find_tile<BM, NTHR>(a.offsets, a.rows, a.E, a.nt, sm_tile, blockIdx.x, t)) return;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, kg = lane >> 4;
  const bool swiglu = a.act == kActSwiglu;
  const int mrows = t.p1 - t.p0, half_n = a.ndim / 2;
  const int n0 = t.nt * (swiglu ? 8 : 16);
  const uint32_t kb = static_cast<uint32_t>(a.kdim) * 2;

  // this lane's row of W and rows of x; past the matrix or the tile: past the
  // resource's end, where loads return zeros
  const int wn = swiglu ? (l16 < 8 ? n0 + l16 : half_n + n0 + l16 - 8) : n0 + l16;
  const bool w_in = swiglu ? n0 + (l16 & 7) < half_n : wn < a.ndim;
  const uint32_t woff = w_in ? static_cast<uint32_t>(wn) * kb + kg * 16 : kMMPastEnd;
  uint32_t xoff[4];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = i * 16 + l16;
    xoff[i] = kMMPastEnd;
    if (r < mrows) {
      const int src = a.slot ? min(max(a.slot[t.p0 + r] / a.topk, 0), a.x_rows - 1) : r;
      xoff[i] = static_cast<uint32_t>(src) * kb + kg * 16;
    }
  }
  const __amdgpu_buffer_rsrc_t w_rs =
      buffer_rsrc(Bb + static_cast<size_t>(t.e) * a.kdim * a.ndim * 2,
                  static_cast<uint32_t>(a.ndim) * kb);
  const __amdgpu_buffer_rsrc_t x_rs =
      a.slot ? buffer_rsrc(Ab, static_cast<uint32_t>(a.x_rows) * kb)
             : buffer_rsrc(Ab + static_cast<size_t>(t.p0) * kb, static_cast<uint32_t>(mrows) * kb);

  f32x4_t acc[4];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // steps of 64 k: two MFMA operands of 32 k each
  const int steps = (a.kdim + 63) / 64;
  frag_t wr[U][2], xr[U][2][MT];
  auto load = [&](int s, frag_t (&w)[2], frag_t (&x)[2][MT]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k0 = s * 64 + h * 32;
      const bool in = k0 + kg * 8 < a.kdim;   // false too for steps past the end
      w[h] = __builtin_bit_cast(frag_t, __builtin_amdgcn_raw_buffer_load_b128(
                 w_rs, in ? woff : kMMPastEnd, in ? k0 * 2 : 0, 0));
#pragma unroll
      for (int i = 0; i < MT; ++i)
        x[h][i] = __builtin_bit_cast(frag_t, __builtin_amdgcn_raw_buffer_load_b128(
                      x_rs, in ? xoff[i] : kMMPastEnd, in ? k0 * 2 : 0, 0));
    }
  };
#pragma unroll
  for (int d = 0; d < U; ++d) load(wv + d * WAVES, wr[d], xr[d]);
  // what is added to the output of piece `it`; the first piece's is requested ahead
  // of the products
  const int out_w = swiglu ? half_n : a.ndim, cols = swiglu ? 8 : 16;
  struct Added {
    uint16_t bias, bias_up, res;
    float res_f;
  };
  auto load_added = [&](int it, Added& v) {
    const int r = it / cols, col = n0 + it - r * cols;
    if (r >= mrows || col >= out_w) return;
    if (a.bias) {
      v.bias = static_cast<const uint16_t*>(a.bias)[col];
      if (swiglu) v.bias_up = static_cast<const uint16_t*>(a.bias)[half_n + col];
    }
    if (a.residual) {
      const size_t at = (static_cast<size_t>(t.p0) + r) * out_w + col;
      if (a.c_f32) v.res_f = static_cast<const float*>(a.residual)[at];
      else v.res = static_cast<const uint16_t*>(a.residual)[at];
    }
  };
  Added add;
  load_added(tid, add);
  for (int s = wv; s < steps; s += U * WAVES) {
#pragma unroll
    for (int d = 0; d < U; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = mfma16x16<T>(wr[d][h], xr[d][h][i], acc[i]);
      load(s + (d + U) * WAVES, wr[d], xr[d]);
    }
  }
  // lane: row l16 of each 16-row part, columns 4 kg + [0, 4)
#pragma unroll
  for (int i = 0; i < MT; ++i)
    *reinterpret_cast<f32x4_t*>(&part[wv][i * 16 + l16][kg * 4]) = acc[i];
  __syncthreads();

  for (int it = tid; it < mrows * cols; it += NTHR) {
    const int r = it / cols, c = it - r * cols, col = n0 + c;
    if (col >= out_w) continue;
    if (it != tid) load_added(it, add);
    const size_t p = static_cast<size_t>(t.p0) + r;
    float v = 0.0f, g = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += part[w][r][c];
    uint16_t* z = static_cast<uint16_t*>(a.z);
    float lo, hi;
    if (a.bias) {
      unpack2<T>(add.bias, lo, hi);
      v += lo;
    }
    if (z) z[p * a.ndim + col] = static_cast<uint16_t>(pack2<T>(v, 0.0f));
    if (swiglu) {
#pragma unroll
      for (int w = 0; w < WAVES; ++w) g += part[w][r][8 + c];
      if (a.bias) {
        unpack2<T>(add.bias_up, lo, hi);
        g += lo;
      }
      if (z) z[p * a.ndim + half_n + col] = static_cast<uint16_t>(pack2<T>(g, 0.0f));
      v = (a.c_f32 ? silu_f32<true>(v) : silu_f32<false>(v)) * g;
    } else {
      v = a.c_f32 ? act_f32<true>(v, a.act) : act_f32<false>(v, a.act);
    }
    const size_t at = p * out_w + col;
    if (a.residual) {
      if (a.c_f32) {
        v += add.res_f;
      } else {
        unpack2<T>(add.res, lo, hi);
        v += lo;
      }
    }
    if (a.c_f32) static_cast<float*>(a.C)[at] = v;
    else static_cast<uint16_t*>(a.C)[at] = static_cast<uint16_t>(pack2<T>(v, 0.0f));
  }
}

// us of a product: blocks of 16 MT rows x 16 columns, `step` per 64 k for the first
// 256 of them and a fifth more for each further 256 (401 x 288 x 2952: 16 rows 10.8
// us timed, 11.0 here; 32 rows 8.9, 9.0; 64 x 64 tiles 12.4), half of it for rows
// that are not there (16 rows of 16 experts x 688 x 1248 6.3, 7.0; 64 x 64 8.9).
// Experts' tiles in more than 1024 blocks stream weights, which the larger tiles do
// better (16 rows of 16 experts x 1536 x 2048: 20.2, 64 x 64 15.7).
inline double mm_few_cost(int mt, int rows, int E, int ndim, int kdim) {
  const double tiles = mm_row_tiles(16 * mt, rows, E), blocks = tiles * ((ndim + 15) / 16);
  if (E != 0 && blocks > 1024) return 1e300;
  if (!mm_fits(mm_most_row_tiles(16 * mt, rows, E) * ((ndim + 15) / 16), 512)) return 1e300;
  const double fill = rows / (tiles * 16 * mt);
  const double step = (mt == 1 ? 0.072 : 0.104) * (0.5 + 0.5 * fill), start = mt == 1 ? 3.4 : 4.2;
  const double rounds = __builtin_ceil(blocks / 256);
  return start + (kdim + 63) / 64 * step * (1.0 + 1.2 * (rounds - 1)) + 0.5 * (rounds - 1);
}

template <class T, int MT, int WAVES, int U>
hipError_t mm_few_launch(MMArgs a, hipStream_t s, bool check) {
  const bool swiglu = a.act == kActSwiglu;
  a.nt = swiglu ? (a.ndim / 2 + 7) / 8 : (a.ndim + 15) / 16;
  const long long tiles = mm_most_row_tiles(16 * MT, a.rows, a.offsets ? a.E : 0) * a.nt;
  const long long grid = (tiles + 7) / 8 * 8;
  if (grid == 0) return hipSuccess;
  if (!mm_fits(grid, WAVES * 64)) return hipErrorInvalidConfiguration;
  if (check) return hipSuccess;
  hipLaunchKernelGGL((mm_few_kernel<T, MT, WAVES, U>), dim3(static_cast<unsigned>(grid)),
                     dim3(WAVES * 64), 0, s, static_cast<const uint8_t*>(a.A),
                     static_cast<const uint8_t*>(a.B), a);
  return hipGetLastError();
}

}  // namespace moe
