// Forward products of int8 operands (moe_linear_w8a8): y = act(z) + residual with
// z = (sum_k q_tk w_nk) s_t u_n + b_n, on the tile and few-row kernels of the 16-bit
// products (mm.h, mm_few.h). Bytes and matrix time of K codes are those of K / 2
// 16-bit values, so the choice of a kernel is theirs for that K.
#include "launch_block.h"
#include "launch_int8.h"
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

hipError_t launch_linear_w8a8(const LinearI8& l, hipStream_t s, bool check) {
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
  const int plan = mm_forward_plan(l.rows, 0, l.N, l.K / 2, l.act);
  return l.y_type == 1 ? launch<i8_tag<fp16_tag>>(a, plan, s, check)
                       : launch<i8_tag<bf16_tag>>(a, plan, s, check);
}

}  // namespace moe
