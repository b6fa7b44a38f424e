// The whole routed layer on int8 weights in one call (moe_layer_w8a8).
#include "launch.h"
#include "launch_block.h"
#include "layer_rows.h"
#include "launch_int8.h"
#include "mm_launch.h"
#include "norm_rows.h"

namespace moe {
namespace {

// out[t] = residual[t] + sum_j w[t, j] y[slot_pos[t k + j]] in increasing j, 8 columns
// a thread (combine.hip, with a residual and the type of the results). slot_pos NULL: y is
// by slot.
template <class T, bool F32>
__global__ __launch_bounds__(256) void combine_out_kernel(const float* __restrict__ y,
                                                          const int* __restrict__ slot_pos,
                                                          const float* __restrict__ w,
                                                          const void* residual, int tokens, int H,
                                                          int k, void* out) {
  constexpr int kJB = 8;
  const int chunks = H / 8;
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= static_cast<long long>(tokens) * chunks) return;
  const int t = static_cast<int>(idx / chunks), c = static_cast<int>(idx % chunks);
  const size_t at = static_cast<size_t>(t) * H + c * 8;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0}, res[8];
  if (residual) row_load8<T>(residual, at, F32, res);
  for (int j0 = 0; j0 < k; j0 += kJB) {
    float wj[kJB], v[kJB][8];
#pragma unroll
    for (int u = 0; u < kJB; ++u) {   // past the last pick: the last again, unused
      const int j = t * k + min(j0 + u, k - 1);
      wj[u] = w[j];
      row_load8<T>(y, static_cast<size_t>(slot_pos ? slot_pos[j] : j) * H + c * 8, true, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kJB; ++u)
      if (j0 + u < k)
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] += wj[u] * v[u][x];
  }
  if (residual)
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] += res[x];
  row_store8<T>(out, at, F32, acc);
}

hipError_t launch_combine_out(const float* y, const int* slot_pos, const float* w,
                              const void* residual, int T, int H, int k, void* out, int out_type,
                              hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(T) * (H / 8) + 255) / 256);
  if (out_type == 2) combine_out_kernel<bf16_tag, true><<<blocks, 256, 0, s>>>(y, slot_pos, w, residual, T, H, k, out);
  else if (out_type == 1) combine_out_kernel<fp16_tag, false><<<blocks, 256, 0, s>>>(y, slot_pos, w, residual, T, H, k, out);
  else combine_out_kernel<bf16_tag, false><<<blocks, 256, 0, s>>>(y, slot_pos, w, residual, T, H, k, out);
  return hipGetLastError();
}

// Workspace of the separate steps: what moe_permute writes, the rows' codes, y.
struct Ws {
  int *offsets, *sorted, *pos, *active, *n_active;
  void* permute;
  int8_t* xq;
  float* xs;
  float* h;
  int8_t* hq;
  float* hs;
  float* y;
  FewRecord* record;
  RowsRecord* rows_record;
  size_t total;
};
Ws carve(void* base, int T, int H, int I, int E, int k) {
  const size_t R = static_cast<size_t>(T) * k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    at += align_up(bytes, 256);
    return p;
  };
  Ws w;
  w.offsets = reinterpret_cast<int*>(take((E + 1) * size_t{4}));
  w.sorted = reinterpret_cast<int*>(take(R * 4));
  w.pos = reinterpret_cast<int*>(take(R * 4));
  w.active = reinterpret_cast<int*>(take(E * size_t{4}));
  w.n_active = reinterpret_cast<int*>(take(4));
  w.permute = take(permute_workspace_bytes(T, E, k));
  w.xq = reinterpret_cast<int8_t*>(take(static_cast<size_t>(T) * H));
  w.xs = reinterpret_cast<float*>(take(T * size_t{4}));
  w.h = reinterpret_cast<float*>(take(R * I * 4));
  w.hq = reinterpret_cast<int8_t*>(take(R * I));
  w.hs = reinterpret_cast<float*>(take(R * 4));
  w.y = reinterpret_cast<float*>(take(R * H * 4));
  w.record = reinterpret_cast<FewRecord*>(take(sizeof(FewRecord)));
  w.rows_record = reinterpret_cast<RowsRecord*>(take(sizeof(RowsRecord)));
  w.total = at;
  return w;
}

// LDS of the few-token kernels: the waves' rings, the codes of all rows, and for the down
// kernel y of the block's tiles.
template <int D>
size_t few_lds(int kind, int T, int H, int I, int k) {
  const size_t ring = kFewWaves * D * kFewSlot, R = static_cast<size_t>(T) * k;
  if (kind == 0) return ring + static_cast<size_t>(T) * (H + 16);
  return ring + R * (I + 16) + static_cast<size_t>((H / 8 + kFewBlocks - 1) / kFewBlocks) * R * 32;
}
constexpr int kFewLds = 160 * 1024 - 11520;   // beside the static arrays

template <int KIND, bool CODES, class T, bool OUT32, int S, int D>
hipError_t few_go(const FewArgs& a, hipStream_t s) {
  auto* kern = &layer_few_kernel<KIND, CODES, T, OUT32, S, D>;
  static MMReady ready;
  const hipError_t e = ready.set(reinterpret_cast<const void*>(kern), kFewLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(kFewBlocks), dim3(kFewThreads), few_lds<D>(KIND, a.T, a.H, a.I, a.k), s, a);
  return hipGetLastError();
}
// Gate/up that makes its codes has 8 always: the lower depths are compiled for it and not
// taken.
int few_depth(int kind, int T, int H, int I, int k) {
  return few_lds<8>(kind, T, H, I, k) <= size_t{kFewLds}   ? 8
         : few_lds<4>(kind, T, H, I, k) <= size_t{kFewLds} ? 4
         : few_lds<2>(kind, T, H, I, k) <= size_t{kFewLds} ? 2 : 0;
}
template <int KIND, bool CODES, class T, bool OUT32, int S>
hipError_t few_at(const FewArgs& a, int depth, hipStream_t s) {
  if (depth == 8) return few_go<KIND, CODES, T, OUT32, S, 8>(a, s);
  if (depth == 4) return few_go<KIND, CODES, T, OUT32, S, 4>(a, s);
  return few_go<KIND, CODES, T, OUT32, S, 2>(a, s);
}
template <class T, int S>
hipError_t few_gateup(const FewArgs& a, const LayerI8Half& p, hipStream_t s) {
  if (p.makes_codes) return few_at<0, false, T, false, S>(a, p.take, s);
  layer_route_kernel<T, S><<<a.T + (a.T + 3) / 4, 256, 0, s>>>(a, const_cast<int8_t*>(a.xq), const_cast<float*>(a.xs));
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : few_at<0, true, bf16_tag, false, 1>(a, p.take, s);
}
template <class T, bool OUT32>
hipError_t few_down(const FewArgs& a, const LayerI8Half& p, hipStream_t s) {
  if (p.makes_codes) return few_at<1, false, T, OUT32, 1>(a, p.take, s);
  const hipError_t e = launch_quant_rows(a.h, 2, a.T * a.k, a.I, const_cast<int8_t*>(a.hq), const_cast<float*>(a.hs), s);
  return e != hipSuccess ? e : few_at<1, true, T, OUT32, 1>(a, p.take, s);
}
template <class T>
hipError_t few_up(const FewArgs& a, const LayerI8Half& p, hipStream_t s) {
  return a.E <= 128 ? few_gateup<T, 2>(a, p, s) : a.E <= 256 ? few_gateup<T, 4>(a, p, s) : few_gateup<T, 16>(a, p, s);
}

// Up to 512 picks: those whose codes do not fit in LDS, and more than 16 tokens while
// experts rarely have more than the 16 rows of a unit. 64 tokens x 4096 x 1536, 32 experts
// against tiles: 4 picks (8 an expert) 127 us against 140; 16 experts (16 an expert) 94.5
// against 87.9. 2048 x 768 x 128 experts, 8 of them: 64 tokens 106 against 124, 17 tokens
// 70 against 85. At 8 an expert seven sizes lie between 12 percent better and 8 worse.
bool rows_fit(int T, int E, int k) {
  const int R = T * k;
  return T <= kFewMaxR && R <= kFewMaxR && (T <= kFewTokens || R <= 8 * E);
}
template <int KIND>
hipError_t rows_go(const RowsArgs& a, hipStream_t s) {
  constexpr int kLds = kFewWaves * kRowsDepth * kRowsSlot;
  auto* kern = &layer_rows_kernel<KIND>;
  static MMReady ready;
  const hipError_t e = ready.set(reinterpret_cast<const void*>(kern), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(kFewBlocks), dim3(kFewThreads), kLds, s, a);
  return hipGetLastError();
}
template <class T>
hipError_t route(const FewArgs& a, Ws& w, hipStream_t s) {
  const unsigned blocks = a.T + (a.T + 3) / 4;
  if (a.E <= 128) layer_route_kernel<T, 2><<<blocks, 256, 0, s>>>(a, w.xq, w.xs);
  else if (a.E <= 256) layer_route_kernel<T, 4><<<blocks, 256, 0, s>>>(a, w.xq, w.xs);
  else layer_route_kernel<T, 16><<<blocks, 256, 0, s>>>(a, w.xq, w.xs);
  return hipGetLastError();
}

}  // namespace

LayerI8Plan layer_w8a8_plan(int T, int H, int I, int E, int k) {
  const int R = T * k;
  const int up = few_depth(0, T, H, I, k), down = few_depth(1, T, H, I, k);
  // Codes are made in a product's own launch up to kFewValues values. Of x: 4096 (two tokens
  // of 2048) 25.0 against 26.4 us for the layer with codes made ahead, 14336 118.8 against
  // 119.9, 28672 117.4 against 115.5. Of h: 12288 25.0 against 25.4, 18432 30.8 against 30.1.
  if (T > 0 && T <= kFewTokens && up && down)
    return {kWayRings, {up, T <= kFewWaves && T * H <= kFewValues},
            {down, static_cast<long long>(R) * I <= kFewValues}};
  if (T > 0 && rows_fit(T, E, k)) return {kWayRingsByRows, {kRowsDepth, false}, {kRowsDepth, false}};
  // Products of few rows an expert stream weights, which the low tiles do better; of more
  // rows the 128-row tiles of the grouped FFN do. The layer by low and by 128-row tiles, us,
  // 2048 x 768, 8 of 128 experts: 32 rows an expert 166 and 173, 64 208 and 203, 96 261 and
  // 235, 128 280 and 256, 256 427 and 387; 4096 x 1536, 4 of 16 experts: 16 rows 92 and 96,
  // 64 114 and 120, 96 128 and 126, 128 160 and 154.
  if (R > 96LL * (R < E ? R : E)) return {kWayLargeTiles, {0, false}, {0, false}};
  return {kWayTiles, {mm_forward_plan(R, E, 2 * I, H / 2, kActSwiglu), false},
          {mm_forward_plan(R, E, H, I / 2, 0), false}};
}

size_t layer_w8a8_workspace_bytes(int T, int H, int I, int E, int k) {
  return carve(nullptr, T, H, I, E, k).total;
}

hipError_t launch_layer_w8a8(const LayerI8& l, void* base, hipStream_t s) {
  const int T = l.T, H = l.H, I = l.I, E = l.E, k = l.k;
  Ws w = carve(base, T, H, I, E, k);
  if (l.offsets) w.offsets = l.offsets;
  const FewArgs few = {l.logits, l.x, w.xq, w.xs, w.hq, w.hs, l.w13, l.s13, l.w2, l.s2, l.residual, l.ids, l.w,
                       l.offsets, w.record, w.h, l.out, T, H, I, E, k};
  const LayerI8Plan plan = layer_w8a8_plan(T, H, I, E, k);
  const int R = T * k;
  if (plan.way == kWayRings) {
    const hipError_t e = l.x_type == 1 ? few_up<fp16_tag>(few, plan.up, s) : few_up<bf16_tag>(few, plan.up, s);
    if (e != hipSuccess) return e;
    return l.out_type == 2 ? few_down<bf16_tag, true>(few, plan.down, s)
         : l.out_type == 1 ? few_down<fp16_tag, false>(few, plan.down, s)
                           : few_down<bf16_tag, false>(few, plan.down, s);
  }
  if (plan.way == kWayRingsByRows) {
    hipError_t e = l.x_type == 1 ? route<fp16_tag>(few, w, s) : route<bf16_tag>(few, w, s);
    if (e != hipSuccess) return e;
    e = rows_go<0>({w.xq, w.xs, l.w13, l.s13, l.ids, w.h, l.offsets, w.rows_record, T, R, H, I, E, k}, s);
    if (e != hipSuccess) return e;
    e = launch_quant_rows(w.h, 2, R, I, w.hq, w.hs, s);
    if (e != hipSuccess) return e;
    e = rows_go<1>({w.hq, w.hs, l.w2, l.s2, l.ids, w.y, nullptr, w.rows_record, R, R, I, H, E, k}, s);
    if (e != hipSuccess) return e;
    return launch_combine_out(w.y, nullptr, l.w, l.residual, T, H, k, l.out, l.out_type, s);
  }
  hipError_t e = launch_route_topk(l.logits, T, E, k, l.ids, l.w, s);
  if (e != hipSuccess) return e;
  e = launch_permute(l.ids, T, E, k, w.offsets, w.sorted, w.pos, w.active, w.n_active, w.permute, s);
  if (e != hipSuccess || T == 0) return e;
  e = launch_quant_rows(l.x, l.x_type, T, H, w.xq, w.xs, s);
  if (e != hipSuccess) return e;
  const bool low = plan.way == kWayTiles;
  e = low ? launch_grouped_i8({w.xq, w.xs, l.w13, l.s13, w.offsets, w.sorted, w.h, R, T, k, E, H, 2 * I, true}, s)
          : launch_w8a8_gateup(T, H, I, E, k, w.xq, w.xs, l.w13, l.s13, w.offsets, w.sorted, w.h, nullptr, s);
  if (e != hipSuccess) return e;
  e = launch_quant_rows(w.h, 2, R, I, w.hq, w.hs, s);
  if (e != hipSuccess) return e;
  e = low ? launch_grouped_i8({w.hq, w.hs, l.w2, l.s2, w.offsets, nullptr, w.y, R, R, 1, E, I, H, false}, s)
          : launch_w8a8_down(T, H, I, E, k, w.hq, w.hs, l.w2, l.s2, w.offsets, w.sorted, w.y, nullptr, s);
  if (e != hipSuccess) return e;
  return launch_combine_out(w.y, w.pos, l.w, l.residual, T, H, k, l.out, l.out_type, s);
}

}  // namespace moe
