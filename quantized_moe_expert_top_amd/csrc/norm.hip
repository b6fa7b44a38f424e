// Norms before and after a block, fused with the block's gate and residual
// scale, forward and backward (moe_block_norm, moe_block_norm_backward).
//
//   n = y p w_post, p = 1/sqrt(mean(y^2) + eps);   r' = r + c g n
//   h = r' q w_pre, q = 1/sqrt(mean(r'^2) + eps)
//
// backward, with d = dh w_pre (per element) and sums over a row's H elements:
//   dr  = dr' + q d - r' q^3 sum(d r') / H          dw_pre  = sum_t dh r' q
//   dn  = c g dr;  e = dn w_post
//   dy  = p e - y p^3 sum(e y) / H                  dw_post = sum_t dn y p
//   dg  = c dr n  (summed over tokens or over the row, as the gate broadcasts)
//
// Both are bound by the bytes of the rows: every row is read once and stays in
// registers over its two reductions.
#include "launch_block.h"
#include "norm_rows.h"

namespace moe {
namespace {

// A row is held by WPR waves, NC chunks of 8 per thread; WPR = 1 puts four rows
// in a block.
template <class T, int WPR, int NC, bool STREAM>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void block_norm_kernel(const NormArgs a) {
  constexpr int kRows = WPR == 1 ? 4 : 1, kRowThreads = WPR * kWave;
  __shared__ float red[2][WPR];
  const int rt = WPR == 1 ? (threadIdx.x & (kWave - 1)) : threadIdx.x;
  const int t = blockIdx.x * kRows + (WPR == 1 ? threadIdx.x >> 6 : 0);
  if (t >= a.T) return;   // whole waves; with WPR > 1, whole blocks
  const int C = a.H / 8;
  const size_t row = static_cast<size_t>(t) * a.H;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float r[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = rt + i * kRowThreads;
    if (c < C) row_load8<T>(a.r, row + c * 8, a.r_f32, r[i]);
    else
#pragma unroll
      for (int x = 0; x < 8; ++x) r[i][x] = 0.0f;
  }
  if (a.y) {
    float y[NC][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = rt + i * kRowThreads;
      if (c < C) row_load8<T>(a.y, row + c * 8, a.y_f32, y[i]);
      else
#pragma unroll
        for (int x = 0; x < 8; ++x) y[i][x] = 0.0f;
#pragma unroll
      for (int x = 0; x < 8; ++x) ss += y[i][x] * y[i][x];
    }
    float f = a.scale;
    if (a.gate_kind == 2) f *= load1<T>(a.gate, t);
    if (a.w_post) f *= 1.0f / sqrtf(row_sum<WPR>(ss, red[0]) * inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = rt + i * kRowThreads;
      if (c >= C) continue;
      if (a.w_post) {
        float w[8];
        row_load8<T>(a.w_post, static_cast<size_t>(c) * 8, false, w);
#pragma unroll
        for (int x = 0; x < 8; ++x) y[i][x] *= w[x];
      }
      if (a.gate_kind == 1 || a.gate_kind == 3) {
        float g[8];
        row_load8<T>(a.gate, (a.gate_kind == 3 ? row : 0) + c * 8, false, g);
#pragma unroll
        for (int x = 0; x < 8; ++x) y[i][x] *= g[x];
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) r[i][x] += f * y[i][x];
      if (a.r_out) row_put8<T, STREAM>(a.r_out, row + c * 8, a.r_f32, r[i]);
    }
  }
  if (a.h) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int x = 0; x < 8; ++x) ss += r[i][x] * r[i][x];
    const float q = 1.0f / sqrtf(row_sum<WPR>(ss, red[1]) * inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = rt + i * kRowThreads;
      if (c >= C) continue;
      float w[8];
      row_load8<T>(a.w_pre, static_cast<size_t>(c) * 8, false, w);
#pragma unroll
      for (int x = 0; x < 8; ++x) r[i][x] *= q * w[x];
      row_put8<T, STREAM>(a.h, row + c * 8, false, r[i]);
    }
  }
}

// Sums of three values over a row held by a whole block of W waves. `red` has
// two halves that alternate between calls, so one barrier per call is enough.
template <int W>
__device__ __forceinline__ void block_sum3(float& u, float& v, float& w, float (*red)[3]) {
  u = wave_sum_f32(u);
  v = wave_sum_f32(v);
  w = wave_sum_f32(w);
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x >> 6;
  if (lane == 0) {
    red[wv][0] = u;
    red[wv][1] = v;
    red[wv][2] = w;
  }
  __syncthreads();
  u = v = w = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    u += red[i][0];
    v += red[i][1];
    w += red[i][2];
  }
}

// What one thread holds of a row: a chunk of 8 of each operand.
struct NormChunk {
  float dr[8], y[8], x[8];   // dr', y, r'; x holds e = dn w_post once r' is used up
  uint4 d;                   // dh as it is stored
};
template <class T>
__device__ __forceinline__ void norm_chunk_dh(const NormChunk& v, float (&d)[8]) {
  unpack2<T>(v.d.x, d[0], d[1]);
  unpack2<T>(v.d.y, d[2], d[3]);
  unpack2<T>(v.d.z, d[4], d[5]);
  unpack2<T>(v.d.w, d[6], d[7]);
}
template <class T>
__device__ __forceinline__ void norm_chunk_load(const NormArgs& a, size_t at, bool in, NormChunk& v) {
#pragma unroll
  for (int x = 0; x < 8; ++x) v.dr[x] = v.y[x] = v.x[x] = 0.0f;
  v.d = make_uint4(0, 0, 0, 0);
  if (!in) return;
  if (a.dr_out) row_load8<T>(a.dr_out, at, a.r_f32, v.dr);
  if (a.y) row_load8<T>(a.y, at, a.y_f32, v.y);
  if (a.dh) {
    row_load8<T>(a.r, at, a.r_f32, v.x);
    v.d = ld16(static_cast<const uint16_t*>(a.dh) + at);
  }
}
// What does not change from row to row, as it is stored: held by a thread for each
// of its chunks over all rows.
struct NormWeights {
  uint4 pre, post, gate;   // gate: a channel gate's
};
template <class T>
__device__ __forceinline__ void norm_weights_load(const NormArgs& a, int c, bool in, NormWeights& w) {
  w.pre = w.post = w.gate = make_uint4(0, 0, 0, 0);
  if (!in) return;
  if (a.w_pre) w.pre = ld16(static_cast<const uint16_t*>(a.w_pre) + c * 8);
  if (a.w_post) w.post = ld16(static_cast<const uint16_t*>(a.w_post) + c * 8);
  if (a.gate_kind == 1) w.gate = ld16(static_cast<const uint16_t*>(a.gate) + c * 8);
}
// v.dr becomes the whole gradient of r'
template <class T>
__device__ __forceinline__ void norm_chunk_dr(const NormArgs& a, const NormWeights& wt, float q,
                                              float back, NormChunk& v) {
  if (!a.dh) return;
  float w[8], d[8];
  unpack8<T>(wt.pre, w);
  norm_chunk_dh<T>(v, d);
#pragma unroll
  for (int x = 0; x < 8; ++x) v.dr[x] += q * d[x] * w[x] - v.x[x] * back;
}
template <class T>
__device__ __forceinline__ void norm_chunk_post(const NormArgs& a, const NormWeights& wt, size_t at,
                                                float tg, float (&w)[8], float (&g)[8]) {
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    w[x] = 1.0f;
    g[x] = tg;
  }
  if (a.w_post) unpack8<T>(wt.post, w);
  if (a.gate_kind == 1) unpack8<T>(wt.gate, g);
  if (a.gate_kind == 3) row_load8<T>(a.gate, at, false, g);
}

// Sums over tokens: sum_t dh r' q (dw_pre) and S = sum_t dr y p, with the gate
// inside where it differs by row (token, element). dw_post and the gradient of a
// channel gate are S times what does not depend on the token: c g S and c w_post S.
//
// Rows blockIdx, blockIdx + grid, ...; the sums over tokens stay in registers
// and go to part[blockIdx] at the end, joined in order afterwards. RELOAD: rows
// too wide to stay in registers beside the sums (H > 8192) are read again, from
// L2, in each of the three phases, and the sums live in part[blockIdx] all along.
template <class T, int W, int NC, bool RELOAD, bool STREAM>
__global__ __launch_bounds__(W * 64) void block_norm_backward_kernel(const NormArgs a) {
  constexpr int kThr = W * kWave, kHeld = RELOAD ? 1 : NC;
  __shared__ float red[2][W][3];
  const int C = a.H / 8;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float* part = a.part ? a.part + static_cast<size_t>(blockIdx.x) * 2 * a.H : nullptr;
  float sw_pre[kHeld][8], sy[kHeld][8];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
#pragma unroll
    for (int x = 0; x < 8; ++x) sw_pre[i][x] = sy[i][x] = 0.0f;
  constexpr int kUnroll = RELOAD ? 1 : NC;
  NormWeights wt[kHeld];
  if constexpr (!RELOAD) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * kThr;
      norm_weights_load<T>(a, c, c < C, wt[i]);
    }
  }
  const bool row_gate = a.gate_kind >= 2;

  // the next row is requested before this one's reductions
  constexpr bool kAhead = !RELOAD;
  NormChunk v[2], nx[2];   // kHeld of each (fixed: captured by a lambda)
  auto request = [&](long long t) {
    if constexpr (!RELOAD) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * kThr;
        norm_chunk_load<T>(a, static_cast<size_t>(t) * a.H + c * 8, c < C && t < a.T, nx[i]);
      }
    }
  };
  if constexpr (kAhead) request(blockIdx.x);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = static_cast<size_t>(t) * a.H;
    float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
    if constexpr (!kAhead) request(t);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) v[i] = nx[i];
    if constexpr (kAhead) request(static_cast<long long>(t) + gridDim.x);
#pragma unroll kUnroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * kThr;
      NormChunk& u = v[RELOAD ? 0 : i];
      if constexpr (RELOAD) {
        norm_chunk_load<T>(a, row + c * 8, c < C, u);
        norm_weights_load<T>(a, c, c < C, wt[0]);
      }
      if (c >= C) continue;
      if (a.dh) {
        float w[8], d[8];
        unpack8<T>(wt[RELOAD ? 0 : i].pre, w);
        norm_chunk_dh<T>(u, d);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          s1 += u.x[x] * u.x[x];
          s2 += d[x] * w[x] * u.x[x];
        }
      }
      if (a.y)
#pragma unroll
        for (int x = 0; x < 8; ++x) s3 += u.y[x] * u.y[x];
    }
    block_sum3<W>(s1, s2, s3, red[0]);
    const float q = 1.0f / sqrtf(s1 * inv_h + a.eps);
    const float p = a.w_post ? 1.0f / sqrtf(s3 * inv_h + a.eps) : 1.0f;
    const float back = s2 * inv_h * q * q * q;   // 0 for a row of zeros at any eps
    const float tg = a.gate_kind == 2 ? load1<T>(a.gate, t) : 1.0f;
    float s4 = 0.0f, s5 = 0.0f, s6 = 0.0f;
#pragma unroll kUnroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * kThr;
      NormChunk& u = v[RELOAD ? 0 : i];
      if constexpr (RELOAD) {
        norm_chunk_load<T>(a, row + c * 8, c < C, u);
        norm_weights_load<T>(a, c, c < C, wt[0]);
      }
      if (c >= C) continue;
      norm_chunk_dr<T>(a, wt[RELOAD ? 0 : i], q, back, u);
      const int hi = RELOAD ? 0 : i;   // where this chunk's sums are held
      if (RELOAD && part && t != blockIdx.x) {
        row_load8<T>(part, static_cast<size_t>(c) * 8, true, sw_pre[0]);
        row_load8<T>(part, static_cast<size_t>(a.H) + c * 8, true, sy[0]);
      } else if (RELOAD) {
#pragma unroll
        for (int x = 0; x < 8; ++x) sw_pre[0][x] = sy[0][x] = 0.0f;
      }
      if (a.dh) {
        float d[8];
        norm_chunk_dh<T>(u, d);
#pragma unroll
        for (int x = 0; x < 8; ++x) sw_pre[hi][x] += d[x] * u.x[x] * q;
      }
      row_put8<T, STREAM>(a.dr, row + c * 8, a.r_f32, u.dr);
      if (a.y) {
        float w[8], g[8], dg[8];
        norm_chunk_post<T>(a, wt[RELOAD ? 0 : i], row + c * 8, tg, w, g);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float cd = a.scale * u.dr[x], yp = u.y[x] * p;
          dg[x] = cd * yp * w[x];
          sy[hi][x] += (row_gate ? g[x] * u.dr[x] : u.dr[x]) * yp;
          u.x[x] = cd * g[x] * w[x];     // from here x holds e
          s4 += u.x[x] * u.y[x];
          s5 += dg[x];
        }
        if (a.gate_kind == 3 && a.dgate) row_put8<T, STREAM>(a.dgate, row + c * 8, false, dg);
      }
      if (RELOAD && part) {
        row_store8<T>(part, static_cast<size_t>(c) * 8, true, sw_pre[0]);
        row_store8<T>(part, static_cast<size_t>(a.H) + c * 8, true, sy[0]);
      }
    }
    if (a.y) {
      block_sum3<W>(s4, s5, s6, red[1]);
      const float bk = a.w_post ? s4 * inv_h * p * p * p : 0.0f;
      if (a.dy)
#pragma unroll kUnroll
        for (int i = 0; i < NC; ++i) {
          const int c = threadIdx.x + i * kThr;
          NormChunk& u = v[RELOAD ? 0 : i];
          if (c >= C) continue;
          if constexpr (RELOAD) {
            norm_chunk_load<T>(a, row + c * 8, true, u);
            norm_weights_load<T>(a, c, true, wt[0]);
            norm_chunk_dr<T>(a, wt[RELOAD ? 0 : i], q, back, u);
            float w[8], g[8];
            norm_chunk_post<T>(a, wt[RELOAD ? 0 : i], row + c * 8, tg, w, g);
#pragma unroll
            for (int x = 0; x < 8; ++x) u.x[x] = a.scale * u.dr[x] * g[x] * w[x];
          }
          float o[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) o[x] = p * u.x[x] - u.y[x] * bk;
          row_put8<T, STREAM>(a.dy, row + c * 8, a.y_f32, o);
        }
      if (a.gate_kind == 2 && a.dgate && threadIdx.x == 0) static_cast<float*>(a.dgate)[t] = s5;
    } else {
      __syncthreads();   // the next row writes red[0] again
    }
  }
  if (RELOAD || part == nullptr) return;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = threadIdx.x + i * kThr;
    if (c >= C) continue;
    row_store8<T>(part, static_cast<size_t>(c) * 8, true, sw_pre[i]);
    row_store8<T>(part, static_cast<size_t>(a.H) + c * 8, true, sy[i]);
  }
}

// H <= 512: a wave holds a whole row (NC chunks of 8 per lane), eight rows in
// flight per block and no barrier before the end, where the waves' sums over
// tokens are joined in wave order. (At H 2048 the row and its sums take 240
// registers, and two waves per SIMD do not cover the loads: 167 us for 16381 rows
// against 107 with a row per block of four waves.)
constexpr int kNormWaves = 8;

template <class T, int NC, bool STREAM>
__global__ __launch_bounds__(kNormWaves * 64, NC == 1 ? 4 : 2) void block_norm_backward_wave_kernel(
    const NormArgs a) {
  __shared__ __attribute__((aligned(16))) float join[kNormWaves - 1][NC * 512];
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x >> 6;
  const int C = a.H / 8;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const bool row_gate = a.gate_kind >= 2;
  NormWeights wt[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = lane + i * kWave;
    norm_weights_load<T>(a, c, c < C, wt[i]);
  }
  float sums[2][NC][8];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int x = 0; x < 8; ++x) sums[k][i][x] = 0.0f;

  // 64-bit: the last stride may pass 2^31
  for (long long t = static_cast<long long>(blockIdx.x) * kNormWaves + wv; t < a.T;
       t += static_cast<long long>(gridDim.x) * kNormWaves) {
    const size_t row = static_cast<size_t>(t) * a.H;
    NormChunk v[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + i * kWave;
      norm_chunk_load<T>(a, row + c * 8, c < C, v[i]);
    }
    float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + i * kWave;
      // one chunk's weights at a time: hoisted together they would spill
      __builtin_amdgcn_sched_barrier(0);
      if (c >= C) continue;
      if (a.dh) {
        float w[8], d[8];
        unpack8<T>(wt[i].pre, w);
        norm_chunk_dh<T>(v[i], d);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          s1 += v[i].x[x] * v[i].x[x];
          s2 += d[x] * w[x] * v[i].x[x];
        }
      }
      if (a.y)
#pragma unroll
        for (int x = 0; x < 8; ++x) s3 += v[i].y[x] * v[i].y[x];
    }
    s1 = wave_sum_f32(s1);
    s2 = wave_sum_f32(s2);
    s3 = wave_sum_f32(s3);
    const float q = 1.0f / sqrtf(s1 * inv_h + a.eps);
    const float p = a.w_post ? 1.0f / sqrtf(s3 * inv_h + a.eps) : 1.0f;
    const float back = s2 * inv_h * q * q * q;   // 0 for a row of zeros at any eps
    const float tg = a.gate_kind == 2 ? load1<T>(a.gate, t) : 1.0f;
    float s4 = 0.0f, s5 = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + i * kWave;
      __builtin_amdgcn_sched_barrier(0);
      if (c >= C) continue;
      NormChunk& u = v[i];
      norm_chunk_dr<T>(a, wt[i], q, back, u);
      if (a.dh) {
        float d[8];
        norm_chunk_dh<T>(u, d);
#pragma unroll
        for (int x = 0; x < 8; ++x) sums[0][i][x] += d[x] * u.x[x] * q;
      }
      row_put8<T, STREAM>(a.dr, row + c * 8, a.r_f32, u.dr);
      if (a.y) {
        float w[8], g[8], dg[8];
        norm_chunk_post<T>(a, wt[i], row + c * 8, tg, w, g);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float cd = a.scale * u.dr[x], yp = u.y[x] * p;
          dg[x] = cd * yp * w[x];
          sums[1][i][x] += (row_gate ? g[x] * u.dr[x] : u.dr[x]) * yp;
          u.x[x] = cd * g[x] * w[x];     // from here x holds e
          s4 += u.x[x] * u.y[x];
          s5 += dg[x];
        }
        if (a.gate_kind == 3 && a.dgate) row_put8<T, STREAM>(a.dgate, row + c * 8, false, dg);
      }
    }
    if (a.y) {
      s4 = wave_sum_f32(s4);
      s5 = wave_sum_f32(s5);
      const float bk = a.w_post ? s4 * inv_h * p * p * p : 0.0f;
      if (a.dy)
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = lane + i * kWave;
          if (c >= C) continue;
          float o[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) o[x] = p * v[i].x[x] - v[i].y[x] * bk;
          row_put8<T, STREAM>(a.dy, row + c * 8, a.y_f32, o);
        }
      if (a.gate_kind == 2 && a.dgate && lane == 0) static_cast<float*>(a.dgate)[t] = s5;
    }
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.H;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k > 0) __syncthreads();   // the sums before are read
    if (wv > 0)
#pragma unroll
      for (int i = 0; i < NC; ++i)
        row_store8<T>(join[wv - 1], static_cast<size_t>(lane + i * kWave) * 8, true, sums[k][i]);
    __syncthreads();
    if (wv == 0)
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = lane + i * kWave;
        if (c >= C) continue;
#pragma unroll
        for (int w = 0; w < kNormWaves - 1; ++w) {
          float o[8];
          row_load8<T>(join[w], static_cast<size_t>(c) * 8, true, o);
#pragma unroll
          for (int x = 0; x < 8; ++x) sums[k][i][x] += o[x];
        }
        row_store8<T>(part, static_cast<size_t>(a.H) * k + c * 8, true, sums[k][i]);
      }
  }
}

// part [blocks][2][H] -> dw_pre, dw_post and a channel gate's gradient (those
// that are asked for), sums in block order over 32 runs: few blocks, so what takes
// the time is how many loads each run has one after another (768 parts of 2 x 2048:
// 7.9 us with 8 runs, 5.0 with 32).
template <class T>
__global__ __launch_bounds__(1024) void norm_parts_kernel(const NormArgs a, int parts,
                                                         float* __restrict__ dw_pre,
                                                         float* __restrict__ dw_post,
                                                         float* __restrict__ dgate) {
  __shared__ float red[32][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + tx, which = blockIdx.y;
  if (which == 0 ? dw_pre == nullptr : dw_post == nullptr && dgate == nullptr) return;   // uniform
  const int run = (parts + 31) / 32, p0 = ty * run, p1 = min(p0 + run, parts);
  float v = 0.0f;
  if (col < a.H)
#pragma unroll 8
    for (int p = p0; p < p1; ++p) v += a.part[(static_cast<size_t>(p) * 2 + which) * a.H + col];
  red[ty][tx] = v;
  __syncthreads();
  if (ty != 0 || col >= a.H) return;
#pragma unroll
  for (int y = 1; y < 32; ++y) v += red[y][tx];
  if (which == 0) {
    dw_pre[col] = v;
  } else {
    v *= a.scale;
    if (dw_post) dw_post[col] = parts && a.gate_kind == 1 ? v * load1<T>(a.gate, col) : v;
    if (dgate) dgate[col] = parts && a.w_post ? v * load1<T>(a.w_post, col) : v;
  }
}

template <class T, bool STREAM>
hipError_t forward(const NormArgs& a, hipStream_t s) {
  const int C = a.H / 8;
  const auto four = dim3((a.T + 3) / 4);
  if (C <= 64) block_norm_kernel<T, 1, 1, STREAM><<<four, 256, 0, s>>>(a);
  else if (C <= 256) block_norm_kernel<T, 4, 1, STREAM><<<a.T, 256, 0, s>>>(a);
  else if (C <= 512) block_norm_kernel<T, 4, 2, STREAM><<<a.T, 256, 0, s>>>(a);
  else if (C <= 1024) block_norm_kernel<T, 16, 1, STREAM><<<a.T, 1024, 0, s>>>(a);
  else block_norm_kernel<T, 16, 2, STREAM><<<a.T, 1024, 0, s>>>(a);
  return hipGetLastError();
}

template <class T, bool STREAM>
hipError_t backward(const NormArgs& a, int blocks, hipStream_t s) {
  const int C = a.H / 8;
  if (C <= 64) block_norm_backward_wave_kernel<T, 1, STREAM><<<blocks, kNormWaves * 64, 0, s>>>(a);
  else if (C <= 128) block_norm_backward_kernel<T, 2, 1, false, STREAM><<<blocks, 128, 0, s>>>(a);
  else if (C <= 256) block_norm_backward_kernel<T, 4, 1, false, STREAM><<<blocks, 256, 0, s>>>(a);
  else if (C <= 512) block_norm_backward_kernel<T, 4, 2, false, STREAM><<<blocks, 256, 0, s>>>(a);
  else if (C <= 1024) block_norm_backward_kernel<T, 8, 2, false, STREAM><<<blocks, 512, 0, s>>>(a);
  else block_norm_backward_kernel<T, 16, 2, true, STREAM><<<blocks, 1024, 0, s>>>(a);
  return hipGetLastError();
}

// The forward's operands from row t0 on.
NormArgs rows_from(NormArgs a, int t0, int rows) {
  const size_t at = static_cast<size_t>(t0) * a.H, rb = a.r_f32 ? 4 : 2, yb = a.y_f32 ? 4 : 2;
  auto from = [](auto& p, size_t bytes) {
    using P = typename std::remove_reference<decltype(p)>::type;
    if (p) p = reinterpret_cast<P>(reinterpret_cast<uintptr_t>(p) + bytes);
  };
  from(a.r, at * rb);
  from(a.y, at * yb);
  from(a.r_out, at * rb);
  from(a.h, at * 2);
  if (a.gate_kind >= 2) from(a.gate, (a.gate_kind == 3 ? at : static_cast<size_t>(t0)) * 2);
  a.T = rows;
  return a;
}

bool streams(const NormArgs& a, long long bytes_per_value) {   // rows of whole cache lines
  return static_cast<long long>(a.T) * a.H * bytes_per_value > (32LL << 20) && a.H % 64 == 0;
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, bool fp16, hipStream_t s) {
  const bool stream = streams(a, (a.r_out ? (a.r_f32 ? 4 : 2) : 0) + (a.h ? 2 : 0));
  // one launch holds less than 2^32 threads: 2^21 rows of 1024
  constexpr int kLaunchRows = 1 << 21;
  for (int t0 = 0, left = a.T; left > 0; left -= kLaunchRows, t0 += kLaunchRows) {
    const NormArgs p = rows_from(a, t0, left < kLaunchRows ? left : kLaunchRows);
    const hipError_t e = stream ? (fp16 ? forward<fp16_tag, true>(p, s) : forward<bf16_tag, true>(p, s))
                                : (fp16 ? forward<fp16_tag, false>(p, s) : forward<bf16_tag, false>(p, s));
    if (e != hipSuccess) return e;
    if (left <= kLaunchRows) break;
  }
  return hipSuccess;
}

int norm_backward_blocks(int T, int H) {
  // as many blocks as the registers let the chip hold at once: one more round of
  // a few of them costs as much as the first (16381 x 2048: 768 blocks 107 us,
  // 1024 blocks 139 us)
  if (H <= 512) {   // a wave per row
    const int need = static_cast<int>((static_cast<long long>(T) + kNormWaves - 1) / kNormWaves);
    return need < 512 ? need : 512;
  }
  const int most = H <= 1024 ? 1536 : H <= 2048 ? 768 : H <= 4096 ? 512 : 256;
  return T < most ? T : most;
}

hipError_t launch_block_norm_backward(const NormArgs& a, bool fp16, float* dw_pre, float* dw_post,
                                      float* dgate_channel, hipStream_t s) {
  const int blocks = norm_backward_blocks(a.T, a.H);
  if (a.T > 0) {
    hipError_t e;
    if (streams(a, (a.r_f32 ? 4 : 2) + (a.dy ? (a.y_f32 ? 4 : 2) : 0)))
      e = fp16 ? backward<fp16_tag, true>(a, blocks, s) : backward<bf16_tag, true>(a, blocks, s);
    else
      e = fp16 ? backward<fp16_tag, false>(a, blocks, s) : backward<bf16_tag, false>(a, blocks, s);
    if (e != hipSuccess) return e;
  }
  if (dw_pre || dw_post || dgate_channel) {
    const dim3 grid((a.H + 31) / 32, 2);
    if (fp16) norm_parts_kernel<fp16_tag><<<grid, 1024, 0, s>>>(a, blocks, dw_pre, dw_post, dgate_channel);
    else norm_parts_kernel<bf16_tag><<<grid, 1024, 0, s>>>(a, blocks, dw_pre, dw_post, dgate_channel);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace moe
