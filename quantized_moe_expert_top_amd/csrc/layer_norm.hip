// Layer norms with the residual addition before them, forward and backward
// (moe_layer_norm, moe_layer_norm_backward).
//
//   r' = r + y;   m = mean(r'), p = 1/sqrt(mean((r' - m)^2) + eps)
//   x^ = (r' - m) p;   h = x^ w + b
//
// backward, with d = dh w (per element) and means over a row's H elements:
//   dr = dr' + p (d - mean(d) - x^ mean(d x^))
//   dw = sum_t dh x^,  db = sum_t dh
//
// Both are bound by the bytes of the rows: every row is read once and stays in
// registers over its two reductions, the mean and then the squares of what is left of
// it (the difference of mean(r'^2) and m^2 would lose the digits that a row's mean
// takes). Forward of 8191 x 2048 with a float32 y: 28.8 us, 168 MB at 5.8 TB/s; gradients of
// 16381 x 2048: 53 us, 268 MB at 5.1 (the rows 48, the last sums 4.6).
#include "launch_block.h"
#include "norm_rows.h"

namespace moe {
namespace {

// A row is held by WPR waves, NC chunks of 8 per thread; WPR = 1 puts four rows in a
// block.
template <class T, int WPR, int NC, bool STREAM>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void layer_norm_kernel(const LayerNormArgs a) {
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
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = rt + i * kRowThreads;
      if (c < C) row_load8<T>(a.y, row + c * 8, a.y_f32, y[i]);
      else
#pragma unroll
        for (int x = 0; x < 8; ++x) y[i][x] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = rt + i * kRowThreads;
#pragma unroll
      for (int x = 0; x < 8; ++x) r[i][x] += y[i][x];
      if (a.r_out && c < C) row_put8<T, STREAM>(a.r_out, row + c * 8, a.r_f32, r[i]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int x = 0; x < 8; ++x) s += r[i][x];
  const float mean = row_sum<WPR>(s, red[0]) * inv_h;
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (rt + i * kRowThreads >= C) continue;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      r[i][x] -= mean;
      ss += r[i][x] * r[i][x];
    }
  }
  const float p = 1.0f / sqrtf(row_sum<WPR>(ss, red[1]) * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = rt + i * kRowThreads;
    if (c >= C) continue;
    float w[8], b[8];
    row_load8<T>(a.w, static_cast<size_t>(c) * 8, false, w);
    if (a.b) row_load8<T>(a.b, static_cast<size_t>(c) * 8, false, b);
    else
#pragma unroll
      for (int x = 0; x < 8; ++x) b[x] = 0.0f;
#pragma unroll
    for (int x = 0; x < 8; ++x) r[i][x] = __builtin_fmaf(r[i][x] * p, w[x], b[x]);
    row_put8<T, STREAM>(a.h, row + c * 8, false, r[i]);
  }
}

// Sums of two values over a row held by W waves; `red` is free again after the next
// call's barrier (two slots alternate).
template <int W>
__device__ __forceinline__ void row_sum2(float& u, float& v, float (*red)[2]) {
  u = wave_sum_f32(u);
  v = wave_sum_f32(v);
  if constexpr (W > 1) {
    const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x >> 6;
    if (lane == 0) {
      red[wv][0] = u;
      red[wv][1] = v;
    }
    __syncthreads();
    u = v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      u += red[i][0];
      v += red[i][1];
    }
  }
}

// What a thread holds of a row: a chunk of 8 of each operand, as it is stored.
template <class T, bool R32>
struct LnChunk {
  Row8<T, R32> x, dr;   // r', dr'
  uint4 d;              // dh
};
// LATE: dr' only where it is added (rows too wide to hold it from the start)
template <class T, bool R32, bool LATE>
__device__ __forceinline__ void ln_load(const LayerNormArgs& a, size_t at, bool in, LnChunk<T, R32>& v) {
  v.x.zero();
  v.dr.zero();
  v.d = make_uint4(0, 0, 0, 0);
  if (!in) return;
  v.x.load(a.r, at);
  v.d = ld16(static_cast<const uint16_t*>(a.dh) + at);
  if (!LATE && a.dr_out) v.dr.load(a.dr_out, at);
}

// One row held by W waves (the whole block, or one wave of it): its gradient, and its
// part of the sums over tokens. The rows' values and products stay unpacked over the three
// phases: unpacked in each of them, the arithmetic takes as long as the memory. (Not the
// products of rows too wide for that, NC 4.)
template <class T, int W, int NC, bool R32, bool LATE, bool STREAM>
__device__ __forceinline__ void ln_row(const LayerNormArgs& a, size_t row, int rt, int C, float inv_h,
                                       const uint4 (&wt)[NC], LnChunk<T, R32> (&v)[NC], float (*red)[W][2],
                                       float (&sw)[NC][8], float (&sb)[NC][8]) {
  constexpr int kThr = W * kWave;
  constexpr bool kHold = NC < 4;
  float x[NC][8], dw[kHold ? NC : 1][8];   // r', then r' - mean; dh w
  auto products = [&](int i, float(&p)[8]) {
    float w[8], d[8];
    unpack8<T>(wt[i], w);
    unpack8<T>(v[i].d, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = d[e] * w[e];
  };
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!kHold) __builtin_amdgcn_sched_barrier(0);   // one chunk's at a time: together they would spill
    float(&q)[8] = dw[kHold ? i : 0];
    v[i].x.values(x[i]);
    products(i, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // zeros past the row
      s1 += x[i][e];
      s2 += q[e];
    }
  }
  row_sum2<W>(s1, s2, red[0]);
  const float mean = s1 * inv_h, md = s2 * inv_h;
  float s3 = 0.0f, s4 = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!kHold) __builtin_amdgcn_sched_barrier(0);
    if (rt + i * kThr >= C) continue;
    float(&q)[8] = dw[kHold ? i : 0];
    if (!kHold) products(i, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[i][e] -= mean;
      s3 += x[i][e] * x[i][e];
      s4 += q[e] * x[i][e];
    }
  }
  row_sum2<W>(s3, s4, red[1]);
  const float p = 1.0f / sqrtf(s3 * inv_h + a.eps);
  const float mx = s4 * inv_h * p;   // mean(d x^)
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = rt + i * kThr;
    if (c >= C) continue;
    if (!kHold) __builtin_amdgcn_sched_barrier(0);
    float(&q)[8] = dw[kHold ? i : 0];
    if (!kHold) products(i, q);
    float d[8], dr[8];
    if (LATE && a.dr_out) v[i].dr.load(a.dr_out, row + c * 8);
    v[i].dr.values(dr);
    unpack8<T>(v[i].d, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xh = x[i][e] * p;
      dr[e] = __builtin_fmaf(p, __builtin_fmaf(-xh, mx, q[e] - md), dr[e]);
      sw[i][e] = __builtin_fmaf(d[e], xh, sw[i][e]);
      sb[i][e] += d[e];
    }
    row_put8<T, STREAM>(a.dr, row + c * 8, R32, dr);
  }
}

// Rows blockIdx, blockIdx + grid, ...; the sums over tokens stay in registers and go to
// part[blockIdx] at the end, joined in order afterwards. AHEAD: the next row is
// requested before this one's reductions.
template <class T, int W, int NC, bool R32, bool AHEAD, bool STREAM>
__global__ __launch_bounds__(W * 64) void layer_norm_backward_kernel(const LayerNormArgs a) {
  constexpr int kThr = W * kWave;
  __shared__ float red[2][W][2];
  const int rt = threadIdx.x, C = a.H / 8;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  uint4 wt[NC];
  float sw[NC][8], sb[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = rt + i * kThr;
    wt[i] = c < C ? ld16(static_cast<const uint16_t*>(a.w) + c * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < 8; ++x) sw[i][x] = sb[i][x] = 0.0f;
  }
  LnChunk<T, R32> v[NC], nx[NC];
  auto request = [&](long long t, LnChunk<T, R32> (&to)[NC]) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = rt + i * kThr;
      ln_load<T, R32, !AHEAD>(a, static_cast<size_t>(t) * a.H + c * 8, c < C && t < a.T, to[i]);
    }
  };
  if constexpr (AHEAD) request(blockIdx.x, nx);
  // 64-bit: the last stride may pass 2^31
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < NC; ++i) v[i] = nx[i];
      request(t + gridDim.x, nx);
    } else {
      request(t, v);
    }
    ln_row<T, W, NC, R32, !AHEAD, STREAM>(a, static_cast<size_t>(t) * a.H, rt, C, inv_h, wt, v, red, sw, sb);
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.H;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = rt + i * kThr;
    if (c >= C) continue;
    row_store8<T>(part, static_cast<size_t>(c) * 8, true, sw[i]);
    row_store8<T>(part, static_cast<size_t>(a.H) + c * 8, true, sb[i]);
  }
}

// H <= 512: a wave holds a whole row, eight rows in flight per block and no barrier
// before the end, where the waves' sums over tokens are joined in wave order.
constexpr int kLnWaves = 8;

template <class T, bool R32, bool STREAM>
__global__ __launch_bounds__(kLnWaves * 64) void layer_norm_backward_wave_kernel(const LayerNormArgs a) {
  __shared__ __attribute__((aligned(16))) float join[kLnWaves - 1][512];
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x >> 6;
  const int C = a.H / 8;
  const bool in = lane < C;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  uint4 wt[1] = {in ? ld16(static_cast<const uint16_t*>(a.w) + lane * 8) : make_uint4(0, 0, 0, 0)};
  float sw[1][8], sb[1][8];
#pragma unroll
  for (int x = 0; x < 8; ++x) sw[0][x] = sb[0][x] = 0.0f;
  for (long long t = static_cast<long long>(blockIdx.x) * kLnWaves + wv; t < a.T;
       t += static_cast<long long>(gridDim.x) * kLnWaves) {
    const size_t row = static_cast<size_t>(t) * a.H;
    LnChunk<T, R32> v[1];
    ln_load<T, R32, false>(a, row + lane * 8, in, v[0]);
    ln_row<T, 1, 1, R32, false, STREAM>(a, row, lane, C, inv_h, wt, v, static_cast<float(*)[1][2]>(nullptr), sw, sb);
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.H;
  auto to_part = [&](float(&s)[8], float* to) {
    if (wv > 0) row_store8<T>(join[wv - 1], static_cast<size_t>(lane) * 8, true, s);
    __syncthreads();
    if (wv == 0 && in) {
#pragma unroll
      for (int w = 0; w < kLnWaves - 1; ++w) {
        float o[8];
        row_load8<T>(join[w], static_cast<size_t>(lane) * 8, true, o);
#pragma unroll
        for (int x = 0; x < 8; ++x) s[x] += o[x];
      }
      row_store8<T>(to, static_cast<size_t>(lane) * 8, true, s);
    }
  };
  to_part(sw[0], part);
  __syncthreads();   // those sums are read
  to_part(sb[0], part + a.H);
}

// part [blocks][2][H] -> dw, db (those that are asked for), in block order over 32 runs:
// what takes the time is how many loads each run has one after another.
__global__ __launch_bounds__(1024) void layer_norm_parts_kernel(const float* __restrict__ part, int H,
                                                                int parts, float* __restrict__ dw,
                                                                float* __restrict__ db) {
  __shared__ float red[32][32];
  float* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;   // uniform
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + tx;
  const int run = (parts + 31) / 32, p0 = ty * run, p1 = min(p0 + run, parts);
  float v = 0.0f;
  if (col < H)
#pragma unroll 8
    for (int p = p0; p < p1; ++p) v += part[(static_cast<size_t>(p) * 2 + blockIdx.y) * H + col];
  red[ty][tx] = v;
  __syncthreads();
  if (ty != 0 || col >= H) return;
#pragma unroll
  for (int y = 1; y < 32; ++y) v += red[y][tx];
  out[col] = v;
}

template <class T, bool STREAM>
hipError_t forward(const LayerNormArgs& a, hipStream_t s) {
  const int C = a.H / 8;
  const unsigned four = (static_cast<unsigned>(a.T) + 3) / 4;
  if (C <= 64) layer_norm_kernel<T, 1, 1, STREAM><<<four, 256, 0, s>>>(a);
  else if (C <= 256) layer_norm_kernel<T, 4, 1, STREAM><<<a.T, 256, 0, s>>>(a);
  else if (C <= 512) layer_norm_kernel<T, 4, 2, STREAM><<<a.T, 256, 0, s>>>(a);
  else if (C <= 1024) layer_norm_kernel<T, 16, 1, STREAM><<<a.T, 1024, 0, s>>>(a);
  else layer_norm_kernel<T, 16, 2, STREAM><<<a.T, 1024, 0, s>>>(a);
  return hipGetLastError();
}

template <class T, bool R32, bool STREAM>
hipError_t backward_as(const LayerNormArgs& a, int blocks, hipStream_t s) {
  const int C = a.H / 8;
  if (C <= 64) layer_norm_backward_wave_kernel<T, R32, STREAM><<<blocks, kLnWaves * 64, 0, s>>>(a);
  else if (C <= 128) layer_norm_backward_kernel<T, 2, 1, R32, true, STREAM><<<blocks, 128, 0, s>>>(a);
  else if (C <= 256) layer_norm_backward_kernel<T, 4, 1, R32, true, STREAM><<<blocks, 256, 0, s>>>(a);
  else if (C <= 512) layer_norm_backward_kernel<T, 8, 1, R32, true, STREAM><<<blocks, 512, 0, s>>>(a);
  else if (C <= 1024) layer_norm_backward_kernel<T, 8, 2, R32, true, STREAM><<<blocks, 512, 0, s>>>(a);
  else layer_norm_backward_kernel<T, 8, 4, R32, false, STREAM><<<blocks, 512, 0, s>>>(a);
  return hipGetLastError();
}
template <class T, bool STREAM>
hipError_t backward(const LayerNormArgs& a, int blocks, hipStream_t s) {
  return a.r_f32 ? backward_as<T, true, STREAM>(a, blocks, s) : backward_as<T, false, STREAM>(a, blocks, s);
}

// The forward's operands from row t0 on.
LayerNormArgs rows_from(LayerNormArgs a, int t0, int rows) {
  const size_t at = static_cast<size_t>(t0) * a.H, rb = a.r_f32 ? 4 : 2, yb = a.y_f32 ? 4 : 2;
  a.r = static_cast<const uint8_t*>(a.r) + at * rb;
  if (a.y) a.y = static_cast<const uint8_t*>(a.y) + at * yb;
  if (a.r_out) a.r_out = static_cast<uint8_t*>(a.r_out) + at * rb;
  a.h = static_cast<uint8_t*>(a.h) + at * 2;
  a.T = rows;
  return a;
}

// Results of more than the L2s' 32 MB go past them, where rows are whole cache lines
// (see row_put8).
bool streams(const LayerNormArgs& a, long long bytes_per_value) {
  return static_cast<long long>(a.T) * a.H * bytes_per_value > (32LL << 20) && a.H % 64 == 0;
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, bool fp16, hipStream_t s) {
  const bool stream = streams(a, (a.r_out ? (a.r_f32 ? 4 : 2) : 0) + 2);
  // one launch holds less than 2^32 threads: 2^21 rows of 1024
  constexpr int kLaunchRows = 1 << 21;
  for (int t0 = 0, left = a.T; left > 0; left -= kLaunchRows, t0 += kLaunchRows) {
    const LayerNormArgs p = rows_from(a, t0, left < kLaunchRows ? left : kLaunchRows);
    const hipError_t e = stream ? (fp16 ? forward<fp16_tag, true>(p, s) : forward<bf16_tag, true>(p, s))
                                : (fp16 ? forward<fp16_tag, false>(p, s) : forward<bf16_tag, false>(p, s));
    if (e != hipSuccess) return e;
    if (left <= kLaunchRows) break;
  }
  return hipSuccess;
}

int layer_norm_backward_blocks(int T, int H) {
  // as many blocks as the chip holds well at once (16381 x 2048: 640 blocks 57.8 us, 768
  // 54.1, 1024 58.8)
  if (H <= 512) {   // a wave per row
    const int need = static_cast<int>((static_cast<long long>(T) + kLnWaves - 1) / kLnWaves);
    return need < 512 ? need : 512;
  }
  const int most = H <= 1024 ? 1536 : H <= 2048 ? 768 : H <= 4096 ? 512 : 256;
  // and at least four rows to each past the first 256, whose sums would cost more to join
  // than their rows take (1024 x 2048: 1024 blocks 13.1 us, 768 12.2, 256 10.4)
  const int want = T / 4 > 256 ? T / 4 : T < 256 ? T : 256;
  return want < most ? want : most;
}

hipError_t launch_layer_norm_backward(const LayerNormArgs& a, bool fp16, float* dw, float* db,
                                      hipStream_t s) {
  const int blocks = layer_norm_backward_blocks(a.T, a.H);
  if (a.T > 0) {
    hipError_t e;
    if (streams(a, a.r_f32 ? 4 : 2))
      e = fp16 ? backward<fp16_tag, true>(a, blocks, s) : backward<bf16_tag, true>(a, blocks, s);
    else
      e = fp16 ? backward<fp16_tag, false>(a, blocks, s) : backward<bf16_tag, false>(a, blocks, s);
    if (e != hipSuccess) return e;
  }
  if (!dw && !db) return hipSuccess;
  layer_norm_parts_kernel<<<dim3((a.H + 31) / 32, 2), 1024, 0, s>>>(a.part, a.H, blocks, dw, db);
  return hipGetLastError();
}

}  // namespace moe
