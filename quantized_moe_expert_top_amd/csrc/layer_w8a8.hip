// The whole routed layer on int8 weights in one call (moe_layer_w8a8).
#include "launch.h"
#include "launch_int8.h"
#include "norm_rows.h"

namespace moe {
namespace {

// out[t] = residual[t] + sum_j w[t, j] y[slot_pos[t k + j]] in increasing j, 8 columns
// a thread (combine.hip, with a residual and the type of the results).
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
      row_load8<T>(y, static_cast<size_t>(slot_pos[j]) * H + c * 8, true, v[u]);
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
  w.total = at;
  return w;
}

}  // namespace

size_t layer_w8a8_workspace_bytes(int T, int H, int I, int E, int k) {
  return carve(nullptr, T, H, I, E, k).total;
}

hipError_t launch_layer_w8a8(const LayerI8& l, void* base, hipStream_t s) {
  const int T = l.T, H = l.H, I = l.I, E = l.E, k = l.k;
  Ws w = carve(base, T, H, I, E, k);
  if (l.offsets) w.offsets = l.offsets;
  hipError_t e = launch_route_topk(l.logits, T, E, k, l.ids, l.w, s);
  if (e != hipSuccess) return e;
  e = launch_permute(l.ids, T, E, k, w.offsets, w.sorted, w.pos, w.active, w.n_active, w.permute, s);
  if (e != hipSuccess || T == 0) return e;
  e = launch_quant_rows(l.x, l.x_type, T, H, w.xq, w.xs, s);
  if (e != hipSuccess) return e;
  e = launch_w8a8_gateup(T, H, I, E, k, w.xq, w.xs, l.w13, l.s13, w.offsets, w.sorted, w.h, nullptr, s);
  if (e != hipSuccess) return e;
  e = launch_quant_rows(w.h, 2, T * k, I, w.hq, w.hs, s);
  if (e != hipSuccess) return e;
  e = launch_w8a8_down(T, H, I, E, k, w.hq, w.hs, l.w2, l.s2, w.offsets, w.sorted, w.y, nullptr, s);
  if (e != hipSuccess) return e;
  return launch_combine_out(w.y, w.pos, l.w, l.residual, T, H, k, l.out, l.out_type, s);
}

}  // namespace moe
