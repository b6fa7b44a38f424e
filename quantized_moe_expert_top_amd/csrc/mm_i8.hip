// Forward products of int8 operands (moe_linear_w8a8): y = act(z) + residual with
// z = (sum_k q_tk w_nk) s_t u_n + b_n, on the tile and few-row kernels of the 16-bit
// products (mm.h, mm_few.h). Bytes and matrix time of K codes are those of K / 2
// 16-bit values, so the choice of a kernel is theirs for that K. 8192 x 7168 -> SwiGLU
// 4096: 206 us, 2.33 POP/s; the matrix pipes are busy 61% of that at 1.78 GHz and the waves
// wait for 29% of their life, so the waits bound it, not the pipes' rate (a plain library
// product of these sizes reaches 2.18, 16384^2 x 8192 2.41, register operands alone 4.2).
#include "launch_block.h"
#include "launch_int8.h"
#include "linear_few.h"
#include "mm_few.h"
#include "mm_launch.h"

namespace moe {
namespace {

template <class T>
hipError_t launch(const MMArgs& a, int plan, hipStream_t s, bool check) {
  switch (plan) {
    case 0: return mm_launch<T, kModeNT, MMBig>(a, s, check);
    case 1: return mm_launch<T, kModeNT, MMMid>(a, s, check);
    case 2: return mm_launch<T, kModeNT, MMWide>(a, s, check);
    case 3: return mm_launch<T, kModeNT, MMSmall>(a, s, check);
    case 4: return mm_launch<T, kModeNT, MMLong>(a, s, check);
    case 5: return mm_launch<T, kModeNT, MMDeep>(a, s, check);
    case 6: return mm_few_launch<T, 1, 8, 2>(a, s, check);
    default: return mm_few_launch<T, 2, 8, 2>(a, s, check);
  }
}

}  // namespace

hipError_t launch_grouped_i8(const GroupedI8& g, hipStream_t s) {
  MMArgs a = {};
  a.A = g.q;
  a.B = g.w;
  a.a_scale = g.q_scale;
  a.b_scale = g.w_scale;
  a.offsets = g.offsets;
  a.slot = g.slot;
  a.x_rows = g.q_rows;
  a.topk = g.topk;
  a.C = g.out;
  a.rows = g.rows;
  a.E = g.E;
  a.splits = 1;
  a.ndim = g.N;
  a.kdim = g.K / 2;
  a.act = g.swiglu ? kActSwiglu : 0;
  a.c_f32 = 1;
  return launch<i8_tag<bf16_tag>>(a, mm_forward_plan(g.rows, g.E, g.N, g.K / 2, a.act), s, false);
}

// ---- up to 16 rows: linear_few.h
namespace {

// LDS of linear_few_kernel beside its static arrays: 8 tiles of 16 x 17 sums and the rows' scales
constexpr int kLinearLds = 160 * 1024 - 9216;
inline long long linear_lds(int depth, int rows, int K) {
  return static_cast<long long>(kFewWaves) * depth * kFewSlot + static_cast<long long>(rows) * (K + 16);
}
template <bool VALUES, class XT, class O, bool OUT32, int D>
hipError_t few_go(const LinearI8& l, const void* x, hipStream_t s) {
  auto* kern = &linear_few_kernel<VALUES, XT, O, OUT32, D>;
  static MMReady ready;
  const hipError_t e = ready.set(reinterpret_cast<const void*>(kern), kLinearLds);
  if (e != hipSuccess) return e;
  const int tiles = l.act == kActSwiglu ? (l.N / 2 + 7) / 8 : (l.N + 15) / 16;
  hipLaunchKernelGGL(kern, dim3(tiles < kFewBlocks ? tiles : kFewBlocks), dim3(kFewThreads),
                     static_cast<size_t>(linear_lds(D, l.rows, l.K)), s, l, x);
  return hipGetLastError();
}
// Rows of values whose codes the block makes leave room for 8: the lower depth is compiled
// for them and not taken.
inline int ring_depth(int rows, int K) { return linear_lds(8, rows, K) <= kLinearLds ? 8 : 4; }
template <bool VALUES, class XT, class O, bool OUT32>
hipError_t few_depth(const LinearI8& l, const void* x, hipStream_t s) {
  if (ring_depth(l.rows, l.K) == 8) return few_go<VALUES, XT, O, OUT32, 8>(l, x, s);
  return few_go<VALUES, XT, O, OUT32, 4>(l, x, s);
}
template <bool VALUES, class XT>
hipError_t few_out(const LinearI8& l, const void* x, hipStream_t s) {
  if (l.y_type == 2) return few_depth<VALUES, XT, bf16_tag, true>(l, x, s);
  return l.y_type == 1 ? few_depth<VALUES, XT, fp16_tag, false>(l, x, s)
                       : few_depth<VALUES, XT, bf16_tag, false>(l, x, s);
}

}  // namespace

LinearI8Plan linear_w8a8_plan(int rows, int K, int N, int act) {
  const long long tiles = act == kActSwiglu ? N / 16 : (N + 15) / 16;
  // The codes of values are made in the product's launch as far as its registers hold the
  // values (kFewValues): 1 x 2048 -> 2048 4.8 us against 7.1 with a launch before it, 2 x
  // 7168 -> SwiGLU 4096 9.0 against 10.8, 16 x 1024 -> 2048 6.9 against 7.1.
  if (rows <= kFewTokens && tiles <= static_cast<long long>(kFewBlocks) * kLinearTiles &&
      linear_lds(4, rows, K) <= kLinearLds)
    return {kPlanRings, ring_depth(rows, K), static_cast<long long>(rows) * K <= kFewValues};
  int plan = mm_forward_plan(rows, 0, N, K / 2, act);
  // Two tiles of 32 rows over all CUs and more: their second round takes as long as the
  // first, however few rows it has (33 x 4096 x 7168, SwiGLU: 22.8 us, tiles of 64 x 64
  // 14.2; 32 rows, one tile: 13.1 against 13.3).
  if (plan == 7 && rows > 32 && mm_row_tiles(32, rows, 0) * ((N + 15) / 16) > kFewBlocks)
    plan = mm_pick_rows(rows, 0, N, K / 2, act).geom;
  return {plan, 0, false};
}
hipError_t launch_linear_w8a8_values(const LinearI8& l, const void* x, int x_type, hipStream_t s) {
  return x_type == 1 ? few_out<true, fp16_tag>(l, x, s) : few_out<true, bf16_tag>(l, x, s);
}

hipError_t launch_linear_w8a8(const LinearI8& l, const LinearI8Plan& plan, hipStream_t s, bool check) {
  if (plan.kernel == kPlanRings) return check ? hipSuccess : few_out<false, bf16_tag>(l, nullptr, s);
  MMArgs a = {};
  a.A = l.q;
  a.B = l.w;
  a.a_scale = l.q_scale;
  a.b_scale = l.w_scale;
  a.bias = l.bias;
  a.residual = l.residual;
  a.C = l.y;
  a.rows = l.rows;
  a.E = 1;
  a.splits = 1;
  a.ndim = l.N;
  a.kdim = l.K / 2;
  a.act = l.act;
  a.c_f32 = l.y_type == 2;
  return l.y_type == 1 ? launch<i8_tag<fp16_tag>>(a, plan.kernel, s, check)
                       : launch<i8_tag<bf16_tag>>(a, plan.kernel, s, check);
}

}  // namespace moe
