// libmoe C ABI, block operators (moe_block.h): argument validation, workspace
// layout, dispatch. As in api.cpp every check runs on the host before anything
// is enqueued, and nothing here allocates or synchronizes.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/moe_block.h"
#include "api_util.h"
#include "launch_block.h"
#include "mm.h"

namespace {

using moe_api::check_device;
using moe_api::fail;
using moe_api::launched;

constexpr int64_t kMaxFeatures = 1 << 20;    // K and N: 32-bit offsets inside a tile's rows
constexpr int64_t kMaxResource = 1LL << 30;  // values behind one buffer resource (2 GiB)
constexpr int32_t kMaxRows = INT32_MAX - 65535;   // room for the ends of tiles and splits
constexpr int64_t kMaxValues = 1LL << 38;    // values of one array: bounds every grid

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

int out_width(const moe_mm_shape* s) { return s->act == MOE_ACT_SWIGLU ? s->N / 2 : s->N; }

moe_status check_mm(const moe_mm_shape* s, bool grouped) {
  if (!s) return fail(MOE_EINVAL, "shape is NULL");
  if (s->rows < 0) return fail(MOE_EINVAL, "rows = %d < 0", s->rows);
  if (s->rows > kMaxRows) return fail(MOE_ESHAPE, "rows = %d above %d", s->rows, kMaxRows);
  if (s->dtype != MOE_BF16 && s->dtype != MOE_FP16)
    return fail(MOE_EINVAL, "dtype = %d is neither MOE_BF16 nor MOE_FP16", s->dtype);
  if (s->act < MOE_ACT_NONE || s->act > MOE_ACT_SWIGLU)
    return fail(MOE_EINVAL, "act = %d is not a MOE_ACT_* value", s->act);
  const int nmod = s->act == MOE_ACT_SWIGLU ? 16 : 8;
  if (s->K < 8 || s->K % 8 || s->K > kMaxFeatures)
    return fail(MOE_ESHAPE, "K = %d must be a positive multiple of 8, at most %d", s->K,
                static_cast<int>(kMaxFeatures));
  if (s->N < nmod || s->N % nmod || s->N > kMaxFeatures)
    return fail(MOE_ESHAPE, "N = %d must be a positive multiple of %d, at most %d", s->N, nmod,
                static_cast<int>(kMaxFeatures));
  if (static_cast<int64_t>(s->N) * s->K > kMaxResource)
    return fail(MOE_ESHAPE, "N*K = %lld above 2^30", static_cast<long long>(s->N) * s->K);
  if (grouped && (s->E < 1 || s->E > MOE_MAX_EXPERTS))
    return fail(MOE_ESHAPE, "E = %d outside [1, %d]", s->E, MOE_MAX_EXPERTS);
  const int64_t wide = s->N > s->K ? s->N : s->K;
  if (s->rows * wide > kMaxValues)
    return fail(MOE_ESHAPE, "rows*max(N, K) = %lld above 2^38", static_cast<long long>(s->rows * wide));
  return MOE_OK;
}

moe_status check_out_type(int32_t type, int32_t dtype, const char* name) {
  if (type != dtype && type != MOE_F32)
    return fail(MOE_EINVAL, "%s = %d is neither dtype (%d) nor MOE_F32", name, type, dtype);
  return MOE_OK;
}

moe_status check_gather(const moe_mm_shape* s, const int32_t* sorted_slot) {
  if (!sorted_slot) return MOE_OK;
  REQUIRE_PTR(sorted_slot);
  if (s->topk < 1) return fail(MOE_ESHAPE, "topk = %d < 1", s->topk);
  if (s->x_rows < 1) return fail(MOE_EINVAL, "x_rows = %d < 1", s->x_rows);
  if (static_cast<int64_t>(s->x_rows) * s->K > kMaxResource)
    return fail(MOE_ESHAPE, "x_rows*K = %lld above 2^30",
                static_cast<long long>(s->x_rows) * s->K);
  return MOE_OK;
}

// Arrays of a call: no output may overlap an input or another output.
struct Span {
  const char* name;
  const void* p;
  size_t bytes;
  bool out;
};
template <int N>
moe_status check_overlap(const Span (&s)[N]) {
  for (int i = 0; i < N; ++i) {
    if (!s[i].out || !s[i].p || !s[i].bytes) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p), b = a + s[i].bytes;
    for (int j = 0; j < N; ++j) {
      if (j == i || (s[j].out && j < i) || !s[j].p || !s[j].bytes) continue;
      const uintptr_t c = reinterpret_cast<uintptr_t>(s[j].p), d = c + s[j].bytes;
      if (a < d && c < b) return fail(MOE_EINVAL, "%s overlaps %s in memory", s[i].name, s[j].name);
    }
  }
  return MOE_OK;
}
size_t values(int64_t rows, int64_t cols, int type) {
  return static_cast<size_t>(rows) * cols * (type == MOE_F32 ? 4 : 2);
}

moe::MMArgs mm_args(const moe_mm_shape* s, const int32_t* offsets, const int32_t* slot) {
  moe::MMArgs a = {};
  a.offsets = offsets;
  a.slot = slot;
  a.rows = s->rows;
  a.x_rows = s->x_rows;
  a.topk = s->topk;
  a.E = offsets ? s->E : 1;
  a.splits = 1;
  return a;
}

// The sizes' last check, before anything is enqueued: what a launch's check returned.
moe_status too_large(hipError_t check) {
  if (check == hipSuccess) return MOE_OK;
  return fail(MOE_ESHAPE, "a launch of these sizes would hold 2^32 threads or more");
}

moe_status run_forward(const moe::MMArgs& a, const moe_mm_shape* s, void* stream, const char* what) {
  const int plan = moe::mm_forward_plan(s->rows, a.offsets ? s->E : 0, s->N, s->K, s->act);
  const bool fp16 = s->dtype == MOE_FP16;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  moe_status r = too_large(moe::launch_mm_nt(a, plan, fp16, st, true));
  if (r || (r = check_device()) != MOE_OK) return r;
  return launched(moe::launch_mm_nt(a, plan, fp16, st, false), what);
}

// Workspace of the gradients: dz, the bias sums' strips, the split products. Grows
// with the rows.
struct MMWs {
  size_t dz, strips, parts, total;
};
MMWs mm_workspace(const moe_mm_shape* s, bool grouped) {
  MMWs w = {};
  size_t at = 0;
  w.dz = at;
  if (!grouped || s->act != MOE_ACT_NONE)
    at += align256(static_cast<size_t>(s->rows) * s->N * 2);
  w.strips = at;
  if (!grouped) at += align256(static_cast<size_t>(moe::dz_most_strips(s->rows, s->N, s->act)) * s->N * 4);
  w.parts = at;
  w.total = at + moe::mm_backward_parts(s->rows, grouped ? s->E : 0, s->N, s->K);
  return w;
}

// The launches of dx = dz W and dw = dz^T x on a given dz, and of `sum` (may be empty).
struct Products {
  moe::MMBackwardPlan plan;
  bool fp16;
  moe::MMArgs nn, tn;   // C NULL: not asked for
  moe::SplitSum sum_dx, sum_dw;
  moe::PartSum sum;
};

Products products_backward(const moe_mm_shape* s, const void* dz, const void* x, const void* w,
                           const int32_t* offsets, const int32_t* slot, void* dx, int dx_dtype,
                           void* dw, int dw_dtype, uint8_t* parts, const moe::PartSum& sum) {
  Products p = {moe::mm_backward_plan(s->rows, offsets ? s->E : 0, s->N, s->K), s->dtype == MOE_FP16,
                mm_args(s, offsets, nullptr), mm_args(s, offsets, slot), {}, {}, sum};
  if (s->rows == 0) dx = nullptr;
  moe::MMArgs& nn = p.nn;
  nn.A = dz;
  nn.B = w;
  nn.C = dx;
  nn.ndim = s->K;
  nn.kdim = s->N;
  nn.c_f32 = dx_dtype == MOE_F32;
  moe::MMArgs& tn = p.tn;
  tn.A = dz;
  tn.B = x;
  tn.C = dw;
  tn.mdim = s->N;
  tn.ndim = s->K;
  tn.c_f32 = dw_dtype == MOE_F32;
  if (dw && p.plan.tn_splits > 1) {
    tn.splits = p.plan.tn_splits;
    tn.C = parts;
    tn.c_f32 = 1;
    p.sum_dw = {reinterpret_cast<const float*>(parts), tn.splits, tn.E,
                static_cast<long long>(s->N) * s->K, dw, dw_dtype};
    parts += align256(static_cast<size_t>(tn.E) * tn.splits * s->N * s->K * 4);
  }
  if (dx && p.plan.nn_splits > 1) {
    nn.splits = p.plan.nn_splits;
    nn.C = parts;
    nn.c_f32 = 1;
    p.sum_dx = {reinterpret_cast<const float*>(parts), nn.splits, 1,
                static_cast<long long>(s->rows) * s->K, dx, dx_dtype};
  }
  return p;
}

// check: only whether every launch fits (see too_large).
moe_status run_products(const Products& p, hipStream_t st, bool check) {
  const bool last = p.sum_dx.out || p.sum_dw.out;   // a launch of sums at the end
  hipError_t e = hipSuccess;
  const bool pair = p.nn.C && p.tn.C && p.plan.pair;
  if (pair) {
    e = moe::launch_mm_pair(p.nn, p.tn, last ? moe::PartSum{} : p.sum, p.plan.pair, p.fp16, st, check);
  } else {
    if (p.nn.C) e = moe::launch_mm_nn(p.nn, p.plan.nn, p.fp16, st, check);
    if (e == hipSuccess && p.tn.C) e = moe::launch_mm_tn(p.tn, p.plan.tn, p.fp16, st, check);
  }
  if (check) return too_large(e);
  if (e != hipSuccess) return launched(e, "gradient launch");
  if (pair && !last) return MOE_OK;   // the sum went along
  return launched(moe::launch_sums(p.sum_dx, p.sum_dw, p.sum, st), "gradient sum launch");
}

}  // namespace

extern "C" {

moe_status moe_grouped_mm(const moe_mm_shape* shape, const void* x, const void* w,
                          const int32_t* expert_offsets, const int32_t* sorted_slot, void* z,
                          void* y, int32_t y_dtype, void* stream) {
  moe_status st = check_mm(shape, true);
  if (st) return st;
  if ((st = check_out_type(y_dtype, shape->dtype, "y_dtype"))) return st;
  if (shape->rows == 0) return MOE_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w);
  REQUIRE_PTR(expert_offsets);
  REQUIRE_PTR(y);
  if (z) REQUIRE_PTR(z);
  if ((st = check_gather(shape, sorted_slot))) return st;
  const int t = shape->dtype;
  if ((st = check_overlap({{"y", y, values(shape->rows, out_width(shape), y_dtype), true},
                           {"z", z, values(shape->rows, shape->N, t), true},
                           {"x", x, values(sorted_slot ? shape->x_rows : shape->rows, shape->K, t), false},
                           {"w", w, shape->E * values(shape->N, shape->K, t), false},
                           {"expert_offsets", expert_offsets, (shape->E + 1) * size_t{4}, false},
                           {"sorted_slot", sorted_slot, shape->rows * size_t{4}, false}})))
    return st;
  moe::MMArgs a = mm_args(shape, expert_offsets, sorted_slot);
  a.A = x;
  a.B = w;
  a.z = z;
  a.C = y;
  a.ndim = shape->N;
  a.kdim = shape->K;
  a.act = shape->act;
  a.c_f32 = y_dtype == MOE_F32;
  return run_forward(a, shape, stream, "moe_grouped_mm launch");
}

size_t moe_grouped_mm_backward_workspace(const moe_mm_shape* shape) {
  if (check_mm(shape, true)) return 0;
  return mm_workspace(shape, true).total;
}

moe_status moe_grouped_mm_backward(const moe_mm_shape* shape, const void* dy, const void* x,
                                   const void* w, const void* z, const int32_t* expert_offsets,
                                   const int32_t* sorted_slot, void* dx, int32_t dx_dtype,
                                   void* dw, int32_t dw_dtype, void* ws, size_t ws_bytes,
                                   void* stream) {
  moe_status st = check_mm(shape, true);
  if (st) return st;
  if (!dx && !dw) return fail(MOE_EINVAL, "dx and dw are both NULL");
  if (dx && (st = check_out_type(dx_dtype, shape->dtype, "dx_dtype"))) return st;
  if (dw && (st = check_out_type(dw_dtype, shape->dtype, "dw_dtype"))) return st;
  if (shape->rows == 0 && !dw) return MOE_OK;
  REQUIRE_PTR(expert_offsets);
  if (dx) REQUIRE_PTR(dx);
  if (dw) REQUIRE_PTR(dw);
  if (shape->rows > 0) {
    REQUIRE_PTR(dy);
    if (shape->act != MOE_ACT_NONE) REQUIRE_PTR(z);
    if (dx) REQUIRE_PTR(w);
    if (dw) {
      REQUIRE_PTR(x);
      if ((st = check_gather(shape, sorted_slot))) return st;
    }
  }
  const MMWs need = mm_workspace(shape, true);
  if (need.total > 0) {
    if (ws_bytes < need.total)
      return fail(MOE_EWORKSPACE, "grouped backward workspace %zu < %zu bytes", ws_bytes, need.total);
    REQUIRE_PTR(ws);
  }
  const int t = shape->dtype;
  const int64_t rows = shape->rows;
  if ((st = check_overlap({{"dx", dx, values(rows, shape->K, dx_dtype), true},
                           {"dw", dw, shape->E * values(shape->N, shape->K, dw_dtype), true},
                           {"ws", ws, need.total, true},
                           {"dy", dy, values(rows, out_width(shape), t), false},
                           {"x", dw ? x : nullptr, values(sorted_slot ? shape->x_rows : rows, shape->K, t), false},
                           {"w", w, shape->E * values(shape->N, shape->K, t), false},
                           {"z", z, values(rows, shape->N, t), false},
                           {"expert_offsets", expert_offsets, (shape->E + 1) * size_t{4}, false},
                           {"sorted_slot", sorted_slot, rows * size_t{4}, false}})))
    return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  void* own = shape->act != MOE_ACT_NONE ? base + need.dz : nullptr;   // dz, where it is not dy
  const Products p = products_backward(shape, own ? own : dy, x, w, expert_offsets,
                                       shape->rows > 0 ? sorted_slot : nullptr, dx, dx_dtype, dw,
                                       dw_dtype, base + need.parts, {});
  if ((st = run_products(p, s, true))) return st;
  if ((st = check_device()) != MOE_OK) return st;
  if (own) {
    st = launched(moe::launch_dz(dy, false, z, expert_offsets, shape->E, shape->rows, shape->N,
                                 shape->act, shape->dtype == MOE_FP16, own, nullptr, false, s),
                  "activation gradient launch");
    if (st) return st;
  }
  return run_products(p, s, false);
}

moe_status moe_linear(const moe_mm_shape* shape, const void* x, const void* w, const void* bias,
                      const void* residual, void* z, void* y, int32_t y_dtype, void* stream) {
  moe_status st = check_mm(shape, false);
  if (st) return st;
  if ((st = check_out_type(y_dtype, shape->dtype, "y_dtype"))) return st;
  if (shape->rows == 0) return MOE_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w);
  REQUIRE_PTR(y);
  if (bias) REQUIRE_PTR(bias);
  if (residual) REQUIRE_PTR(residual);
  if (z) REQUIRE_PTR(z);
  const int t = shape->dtype;
  const size_t y_bytes = values(shape->rows, out_width(shape), y_dtype);
  if ((st = check_overlap({{"y", y, y_bytes, true},
                           {"z", z, values(shape->rows, shape->N, t), true},
                           {"x", x, values(shape->rows, shape->K, t), false},
                           {"w", w, values(shape->N, shape->K, t), false},
                           {"bias", bias, values(1, shape->N, t), false},
                           {"residual", residual == y ? nullptr : residual, y_bytes, false}})))
    return st;
  moe::MMArgs a = mm_args(shape, nullptr, nullptr);
  a.A = x;
  a.B = w;
  a.bias = bias;
  a.residual = residual;
  a.z = z;
  a.C = y;
  a.ndim = shape->N;
  a.kdim = shape->K;
  a.act = shape->act;
  a.c_f32 = y_dtype == MOE_F32;
  return run_forward(a, shape, stream, "moe_linear launch");
}

size_t moe_linear_backward_workspace(const moe_mm_shape* shape) {
  if (check_mm(shape, false)) return 0;
  return mm_workspace(shape, false).total;
}

moe_status moe_linear_backward(const moe_mm_shape* shape, const void* dy, int32_t dy_dtype,
                               const void* x, const void* w, const void* z, void* dx,
                               int32_t dx_dtype, void* dw, void* dbias, int32_t dw_dtype, void* ws,
                               size_t ws_bytes, void* stream) {
  moe_status st = check_mm(shape, false);
  if (st) return st;
  if (!dx && !dw && !dbias) return fail(MOE_EINVAL, "dx, dw and dbias are all NULL");
  if ((st = check_out_type(dy_dtype, shape->dtype, "dy_dtype"))) return st;
  if (dx && (st = check_out_type(dx_dtype, shape->dtype, "dx_dtype"))) return st;
  if ((dw || dbias) && (st = check_out_type(dw_dtype, shape->dtype, "dw_dtype"))) return st;
  if (shape->rows == 0 && !dw && !dbias) return MOE_OK;
  if (dx) REQUIRE_PTR(dx);
  if (dw) REQUIRE_PTR(dw);
  if (dbias) REQUIRE_PTR(dbias);
  if (shape->rows > 0) {
    REQUIRE_PTR(dy);
    if (shape->act != MOE_ACT_NONE) REQUIRE_PTR(z);
    if (dx) REQUIRE_PTR(w);
    if (dw) REQUIRE_PTR(x);
  }
  const MMWs need = mm_workspace(shape, false);
  if (need.total > 0) {
    if (ws_bytes < need.total)
      return fail(MOE_EWORKSPACE, "linear backward workspace %zu < %zu bytes", ws_bytes, need.total);
    REQUIRE_PTR(ws);
  }
  const int t = shape->dtype;
  const int64_t rows = shape->rows;
  if ((st = check_overlap({{"dx", dx, values(rows, shape->K, dx_dtype), true},
                           {"dw", dw, values(shape->N, shape->K, dw_dtype), true},
                           {"dbias", dbias, values(1, shape->N, dw_dtype), true},
                           {"ws", ws, need.total, true},
                           {"dy", dy, values(rows, out_width(shape), dy_dtype), false},
                           {"x", x, values(rows, shape->K, t), false},
                           {"w", w, values(shape->N, shape->K, t), false},
                           {"z", z, values(rows, shape->N, t), false}})))
    return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  // dy itself is dz where no activation and no rounding stands between them
  const bool pass = shape->act != MOE_ACT_NONE || dy_dtype == MOE_F32;
  void* own = pass && (dx || dw) ? base + need.dz : nullptr;
  float* strips = dbias ? reinterpret_cast<float*>(base + need.strips) : nullptr;
  const moe::PartSum sum = {strips, dbias ? moe::dz_strips(shape->rows, shape->N, shape->act) : 0,
                            shape->N, dbias, dw_dtype};
  const Products p = products_backward(shape, own ? own : dy, x, w, nullptr, nullptr, dx, dx_dtype,
                                       dw, dw_dtype, base + need.parts, sum);
  if ((st = run_products(p, s, true))) return st;
  if ((st = check_device()) != MOE_OK) return st;
  if (own || dbias) {
    st = launched(moe::launch_dz(dy, dy_dtype == MOE_F32, z, nullptr, 1, shape->rows, shape->N,
                                 shape->act, shape->dtype == MOE_FP16, own, strips,
                                 dw_dtype == MOE_F32, s),
                  "activation gradient launch");
    if (st) return st;
  }
  return run_products(p, s, false);
}

moe_status moe_product_plan(const moe_mm_shape* shape, int32_t grouped, int32_t* plan) {
  const moe_status st = check_mm(shape, grouped != 0);
  if (st) return st;
  if (!plan) return fail(MOE_EINVAL, "plan is NULL");
  const int E = grouped ? shape->E : 0;
  const moe::MMBackwardPlan b = moe::mm_backward_plan(shape->rows, E, shape->N, shape->K);
  const int32_t v[6] = {moe::mm_forward_plan(shape->rows, E, shape->N, shape->K, shape->act),
                        b.pair, b.nn, b.nn_splits, b.tn, b.tn_splits};
  for (int i = 0; i < 6; ++i) plan[i] = v[i];
  return MOE_OK;
}

static moe_status check_norm(const moe_norm_shape* s) {
  if (!s) return fail(MOE_EINVAL, "shape is NULL");
  if (s->T < 0) return fail(MOE_EINVAL, "T = %d < 0", s->T);
  if (s->H < 8 || s->H % 8 || s->H > MOE_NORM_MAX_H)
    return fail(MOE_ESHAPE, "H = %d must be a positive multiple of 8, at most %d", s->H, MOE_NORM_MAX_H);
  if (s->dtype != MOE_BF16 && s->dtype != MOE_FP16)
    return fail(MOE_EINVAL, "dtype = %d is neither MOE_BF16 nor MOE_FP16", s->dtype);
  moe_status st;
  if ((st = check_out_type(s->r_dtype, s->dtype, "r_dtype"))) return st;
  if ((st = check_out_type(s->y_dtype, s->dtype, "y_dtype"))) return st;
  if (s->gate < MOE_GATE_NONE || s->gate > MOE_GATE_ELEMENT)
    return fail(MOE_EINVAL, "gate = %d is not a MOE_GATE_* value", s->gate);
  if (!(s->eps > 0.0f) || !std::isfinite(s->eps)) return fail(MOE_EINVAL, "eps must be positive");
  if (!std::isfinite(s->scale)) return fail(MOE_EINVAL, "scale must be finite");
  return MOE_OK;
}

static size_t gate_bytes(const moe_norm_shape* s) {
  return values(s->gate == MOE_GATE_CHANNEL ? 1 : s->T, s->gate == MOE_GATE_TOKEN ? 1 : s->H, s->dtype);
}

static moe::NormArgs norm_args(const moe_norm_shape* s) {
  moe::NormArgs a = {};
  a.T = s->T;
  a.H = s->H;
  a.gate_kind = s->gate;
  a.r_f32 = s->r_dtype == MOE_F32;
  a.y_f32 = s->y_dtype == MOE_F32;
  a.scale = s->scale;
  a.eps = s->eps;
  return a;
}

moe_status moe_block_norm(const moe_norm_shape* shape, const void* r, const void* y,
                          const void* w_post, const void* gate, const void* w_pre, void* r_out,
                          void* h, void* stream) {
  moe_status st = check_norm(shape);
  if (st) return st;
  if (!r_out && !h) return fail(MOE_EINVAL, "r_out and h are both NULL");
  if (!h != !w_pre) return fail(MOE_EINVAL, "h and w_pre go together");
  if (!y && (w_post || r_out || shape->gate != MOE_GATE_NONE))
    return fail(MOE_EINVAL, "w_post, gate and r_out need y");
  if (shape->T == 0) return MOE_OK;
  REQUIRE_PTR(r);
  if (y) REQUIRE_PTR(y);
  if (w_post) REQUIRE_PTR(w_post);
  if (shape->gate != MOE_GATE_NONE) REQUIRE_PTR(gate);
  if (w_pre) REQUIRE_PTR(w_pre);
  if (r_out) REQUIRE_PTR(r_out);
  if (h) REQUIRE_PTR(h);
  const int64_t T = shape->T, H = shape->H;
  const int t = shape->dtype;
  if ((st = check_overlap({{"r_out", r_out, values(T, H, shape->r_dtype), true},
                           {"h", h, values(T, H, t), true},
                           {"r", r, values(T, H, shape->r_dtype), false},
                           {"y", y, values(T, H, shape->y_dtype), false},
                           {"w_post", w_post, values(1, H, t), false},
                           {"w_pre", w_pre, values(1, H, t), false},
                           {"gate", shape->gate ? gate : nullptr, gate_bytes(shape), false}})))
    return st;
  if ((st = check_device()) != MOE_OK) return st;
  moe::NormArgs a = norm_args(shape);
  a.r = r;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.r_out = r_out;
  a.h = h;
  return launched(moe::launch_block_norm(a, shape->dtype == MOE_FP16, static_cast<hipStream_t>(stream)),
                  "moe_block_norm launch");
}

size_t moe_block_norm_backward_workspace(int32_t T, int32_t H) {
  if (T < 0 || H < 8 || H % 8 || H > MOE_NORM_MAX_H) return 0;
  return align256(static_cast<size_t>(moe::norm_backward_blocks(T, H)) * 2 * H * 4);
}

moe_status moe_block_norm_backward(const moe_norm_shape* shape, const void* r_out,
                                   const void* dr_out, const void* dh, const void* y,
                                   const void* w_post, const void* gate, const void* w_pre,
                                   void* dr, void* dy, float* dw_post, float* dw_pre, void* dgate,
                                   void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_norm(shape);
  if (st) return st;
  const int T = shape->T, gk = shape->gate;
  if (!dr_out && !dh) return fail(MOE_EINVAL, "dr_out and dh are both NULL");
  if (!dh != !w_pre) return fail(MOE_EINVAL, "dh and w_pre go together");
  if (!y && (w_post || dy || dw_post || dgate || gk != MOE_GATE_NONE))
    return fail(MOE_EINVAL, "w_post, gate and their gradients need y");
  if (dw_post && !w_post) return fail(MOE_EINVAL, "dw_post needs w_post");
  if (dw_pre && !dh) return fail(MOE_EINVAL, "dw_pre needs dh");
  if (dgate && gk == MOE_GATE_NONE) return fail(MOE_EINVAL, "dgate needs a gate");
  float* dg_channel = gk == MOE_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  const bool sums = dw_post || dw_pre || dg_channel;
  if (T == 0 && !sums) return MOE_OK;
  if (dw_post) REQUIRE_PTR(dw_post);
  if (dw_pre) REQUIRE_PTR(dw_pre);
  if (dgate) REQUIRE_PTR(dgate);
  if (T > 0) {
    if (dr_out) REQUIRE_PTR(dr_out);
    if (dh) {
      REQUIRE_PTR(dh);
      REQUIRE_PTR(r_out);
      REQUIRE_PTR(w_pre);
    }
    if (y) REQUIRE_PTR(y);
    if (w_post) REQUIRE_PTR(w_post);
    if (gk != MOE_GATE_NONE) REQUIRE_PTR(gate);
    REQUIRE_PTR(dr);
    if (dy) REQUIRE_PTR(dy);
  }
  const size_t need = moe_block_norm_backward_workspace(T, shape->H);
  if (sums && need > 0) {
    if (ws_bytes < need)
      return fail(MOE_EWORKSPACE, "block norm backward workspace %zu < %zu bytes", ws_bytes, need);
    REQUIRE_PTR(ws);
  }
  const int64_t H = shape->H;
  const int t = shape->dtype;
  if ((st = check_overlap({{"dr", dr, values(T, H, shape->r_dtype), true},
                           {"dy", dy, values(T, H, shape->y_dtype), true},
                           {"dw_post", dw_post, values(1, H, MOE_F32), true},
                           {"dw_pre", dw_pre, values(1, H, MOE_F32), true},
                           {"dgate", dgate, gate_bytes(shape) * (gk == MOE_GATE_ELEMENT ? 1 : 2), true},
                           {"ws", sums ? ws : nullptr, need, true},
                           {"r_out", dh ? r_out : nullptr, values(T, H, shape->r_dtype), false},
                           {"dr_out", dr_out, values(T, H, shape->r_dtype), false},
                           {"dh", dh, values(T, H, t), false},
                           {"y", y, values(T, H, shape->y_dtype), false},
                           {"w_post", w_post, values(1, H, t), false},
                           {"w_pre", w_pre, values(1, H, t), false},
                           {"gate", gk ? gate : nullptr, gate_bytes(shape), false}})))
    return st;
  if ((st = check_device()) != MOE_OK) return st;
  moe::NormArgs a = norm_args(shape);
  a.r = r_out;
  a.dr_out = dr_out;
  a.dh = dh;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.dr = dr;
  a.dy = dy;
  a.dgate = dgate;
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  return launched(moe::launch_block_norm_backward(a, shape->dtype == MOE_FP16, dw_pre, dw_post,
                                                  dg_channel, static_cast<hipStream_t>(stream)),
                  "moe_block_norm_backward launch");
}

moe_status moe_combine_backward(const float* dout, const float* y, const int32_t* slot_pos,
                                const int32_t* topk_ids, const float* topk_w, int32_t T, int32_t H,
                                int32_t E, int32_t k, void* dy, int32_t dy_dtype, float* dtopk_w,
                                float* dlogits, void* stream) {
  if (T < 0) return fail(MOE_EINVAL, "T = %d < 0", T);
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ESHAPE, "E = %d outside [1, %d]", E, MOE_MAX_EXPERTS);
  if (k < 1 || k > E || k > MOE_MAX_TOPK)
    return fail(MOE_ESHAPE, "k = %d outside [1, min(E=%d, %d)]", k, E, MOE_MAX_TOPK);
  if (H < 8 || H % 8) return fail(MOE_ESHAPE, "H = %d must be a positive multiple of 8", H);
  if (static_cast<int64_t>(T) * k >= (1LL << 31))
    return fail(MOE_ESHAPE, "T*k = %lld does not fit int32", static_cast<long long>(T) * k);
  if (!dy && !dtopk_w && !dlogits) return fail(MOE_EINVAL, "dy, dtopk_w and dlogits are all NULL");
  if (dy && dy_dtype != MOE_BF16 && dy_dtype != MOE_FP16 && dy_dtype != MOE_F32)
    return fail(MOE_EINVAL, "dy_dtype = %d is no MOE_BF16, MOE_FP16 or MOE_F32", dy_dtype);
  if (T == 0) return MOE_OK;
  REQUIRE_PTR(dout);
  REQUIRE_PTR(slot_pos);
  REQUIRE_PTR(topk_w);
  if (dtopk_w || dlogits) REQUIRE_PTR(y);
  if (dlogits) REQUIRE_PTR(topk_ids);
  if (dy) REQUIRE_PTR(dy);
  if (dtopk_w) REQUIRE_PTR(dtopk_w);
  if (dlogits) REQUIRE_PTR(dlogits);
  moe_status st;
  const int64_t R = static_cast<int64_t>(T) * k;
  if ((st = check_overlap({{"dy", dy, values(R, H, dy_dtype), true},
                           {"dtopk_w", dtopk_w, values(T, k, MOE_F32), true},
                           {"dlogits", dlogits, values(T, E, MOE_F32), true},
                           {"dout", dout, values(T, H, MOE_F32), false},
                           {"y", dtopk_w || dlogits ? y : nullptr, values(R, H, MOE_F32), false},
                           {"slot_pos", slot_pos, values(R, 1, MOE_F32), false},
                           {"topk_w", topk_w, values(R, 1, MOE_F32), false},
                           {"topk_ids", dlogits ? topk_ids : nullptr, values(R, 1, MOE_F32), false}})))
    return st;
  if ((st = check_device()) != MOE_OK) return st;
  return launched(moe::launch_combine_backward(dout, y, slot_pos, topk_ids, topk_w, T, H, E, k, dy,
                                               dy ? dy_dtype : MOE_F32, dtopk_w, dlogits,
                                               static_cast<hipStream_t>(stream)),
                  "moe_combine_backward launch");
}

}  // extern "C"
