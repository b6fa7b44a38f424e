// libmoe C ABI, int8 operators (moe_int8.h): argument validation, workspaces, dispatch.
// As in api.cpp every check runs on the host before anything is enqueued, and nothing
// here allocates or synchronizes.
#include <hip/hip_runtime.h>

#include "../../include/moe_int8.h"
#include "api_util.h"
#include "launch_int8.h"

namespace {

using moe_api::align256;
using moe_api::check_device;
using moe_api::check_overlap;
using moe_api::fail;
using moe_api::launched;
using moe_api::values;

constexpr int32_t kMaxRows = INT32_MAX - 65535;   // room for the ends of tiles
constexpr int64_t kMaxN = 1 << 20;                // 32-bit offsets inside a tile's rows
constexpr int64_t kMaxWeight = 1LL << 30;         // bytes behind one buffer resource
constexpr int64_t kMaxValues = 1LL << 38;         // values of one array: bounds every grid

bool floating(int32_t t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_F32; }

moe_status check_rows(int32_t rows, int32_t K, int kmod) {
  if (rows < 0) return fail(MOE_EINVAL, "rows = %d < 0", rows);
  if (rows > kMaxRows) return fail(MOE_ESHAPE, "rows = %d above %d", rows, kMaxRows);
  if (K < kmod || K % kmod || K > MOE_INT8_MAX_K)
    return fail(MOE_ESHAPE, "K = %d must be a positive multiple of %d, at most %d", K, kmod,
                MOE_INT8_MAX_K);
  if (static_cast<int64_t>(rows) * K > kMaxValues)
    return fail(MOE_ESHAPE, "rows*K = %lld above 2^38", static_cast<long long>(rows) * K);
  return MOE_OK;
}

moe_status check_linear(const moe_w8_shape* s) {
  if (!s) return fail(MOE_EINVAL, "shape is NULL");
  const moe_status st = check_rows(s->rows, s->K, 16);
  if (st) return st;
  if (s->x_dtype != MOE_INT8 && s->x_dtype != MOE_BF16 && s->x_dtype != MOE_FP16)
    return fail(MOE_EINVAL, "x_dtype = %d is no MOE_INT8, MOE_BF16 or MOE_FP16", s->x_dtype);
  if (!floating(s->y_dtype))
    return fail(MOE_EINVAL, "y_dtype = %d is no MOE_BF16, MOE_FP16 or MOE_F32", s->y_dtype);
  if (s->act < MOE_ACT_NONE || s->act > MOE_ACT_SWIGLU)
    return fail(MOE_EINVAL, "act = %d is not a MOE_ACT_* value", s->act);
  const int nmod = s->act == MOE_ACT_SWIGLU ? 16 : 8;
  if (s->N < nmod || s->N % nmod || s->N > kMaxN)
    return fail(MOE_ESHAPE, "N = %d must be a positive multiple of %d, at most %d", s->N, nmod,
                static_cast<int>(kMaxN));
  if (static_cast<int64_t>(s->N) * s->K > kMaxWeight)
    return fail(MOE_ESHAPE, "N*K = %lld above 2^30", static_cast<long long>(s->N) * s->K);
  if (static_cast<int64_t>(s->rows) * s->N > kMaxValues)
    return fail(MOE_ESHAPE, "rows*N = %lld above 2^38", static_cast<long long>(s->rows) * s->N);
  return MOE_OK;
}

size_t codes_bytes(int32_t rows, int32_t K) { return align256(static_cast<size_t>(rows) * K); }

}  // namespace

extern "C" {

moe_status moe_quant_rows(const void* x, int32_t x_dtype, int32_t rows, int32_t K, int8_t* q,
                          float* scale, void* stream) {
  moe_status st = check_rows(rows, K, 8);
  if (st) return st;
  if (!floating(x_dtype))
    return fail(MOE_EINVAL, "x_dtype = %d is no MOE_BF16, MOE_FP16 or MOE_F32", x_dtype);
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(q);
  REQUIRE_PTR(scale);
  if ((st = check_overlap({{"q", q, values(rows, K, MOE_INT8), true},
                           {"scale", scale, values(rows, 1, MOE_F32), true},
                           {"x", x, values(rows, K, x_dtype), false}})))
    return st;
  if ((st = check_device()) != MOE_OK) return st;
  return launched(moe::launch_quant_rows(x, x_dtype, rows, K, q, scale, static_cast<hipStream_t>(stream)),
                  "moe_quant_rows launch");
}

size_t moe_linear_w8a8_workspace(int32_t rows, int32_t K) {
  if (check_rows(rows, K, 16)) return 0;
  return codes_bytes(rows, K) + align256(static_cast<size_t>(rows) * 4);
}

moe_status moe_linear_w8a8(const moe_w8_shape* s, const void* x, const float* x_scale,
                           const int8_t* w, const float* w_scale, const float* bias,
                           const void* residual, void* y, void* ws, size_t ws_bytes,
                           void* stream) {
  moe_status st = check_linear(s);
  if (st) return st;
  const bool codes = s->x_dtype == MOE_INT8;
  if (!codes && x_scale) return fail(MOE_EINVAL, "x_scale goes with codes (x_dtype MOE_INT8)");
  if (s->rows == 0) return MOE_OK;
  REQUIRE_PTR(x);
  if (codes) REQUIRE_PTR(x_scale);
  REQUIRE_PTR(w);
  REQUIRE_PTR(w_scale);
  if (bias) REQUIRE_PTR(bias);
  if (residual) REQUIRE_PTR(residual);
  REQUIRE_PTR(y);
  const size_t need = codes ? 0 : moe_linear_w8a8_workspace(s->rows, s->K);
  if (need > 0) {
    if (ws_bytes < need)
      return fail(MOE_EWORKSPACE, "linear w8a8 workspace %zu < %zu bytes", ws_bytes, need);
    REQUIRE_PTR(ws);
  }
  const int64_t rows = s->rows, No = s->act == MOE_ACT_SWIGLU ? s->N / 2 : s->N;
  const size_t y_bytes = values(rows, No, s->y_dtype);
  if ((st = check_overlap({{"y", y, y_bytes, true},
                           {"ws", need ? ws : nullptr, need, true},
                           {"x", x, values(rows, s->K, s->x_dtype), false},
                           {"x_scale", x_scale, values(rows, 1, MOE_F32), false},
                           {"w", w, values(s->N, s->K, MOE_INT8), false},
                           {"w_scale", w_scale, values(1, s->N, MOE_F32), false},
                           {"bias", bias, values(1, s->N, MOE_F32), false},
                           {"residual", residual == y ? nullptr : residual, y_bytes, false}})))
    return st;
  moe::LinearI8 l = {};
  l.q = static_cast<const int8_t*>(x);
  l.q_scale = x_scale;
  int8_t* made = static_cast<int8_t*>(ws);
  float* made_scale = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + codes_bytes(s->rows, s->K));
  if (!codes) {
    l.q = made;
    l.q_scale = made_scale;
  }
  l.w = w;
  l.w_scale = w_scale;
  l.bias = bias;
  l.residual = residual;
  l.y = y;
  l.y_type = s->y_dtype;
  l.rows = s->rows;
  l.K = s->K;
  l.N = s->N;
  l.act = s->act;
  const hipStream_t stm = static_cast<hipStream_t>(stream);
  const moe::LinearI8Plan plan = moe::linear_w8a8_plan(s->rows, s->K, s->N, s->act);
  if (moe::launch_linear_w8a8(l, plan, stm, true) != hipSuccess)
    return fail(MOE_ESHAPE, "a launch of these sizes would hold 2^32 threads or more");
  if ((st = check_device()) != MOE_OK) return st;
  if (!codes && plan.makes_codes)
    return launched(moe::launch_linear_w8a8_values(l, x, s->x_dtype, stm), "moe_linear_w8a8 launch");
  if (!codes) {
    st = launched(moe::launch_quant_rows(x, s->x_dtype, s->rows, s->K, made, made_scale, stm),
                  "moe_linear_w8a8 codes launch");
    if (st) return st;
  }
  return launched(moe::launch_linear_w8a8(l, plan, stm, false), "moe_linear_w8a8 launch");
}

moe_status moe_linear_w8a8_plan(const moe_w8_shape* s, int32_t* plan) {
  const moe_status st = check_linear(s);
  if (st) return st;
  if (!plan) return fail(MOE_EINVAL, "plan is NULL");
  const moe::LinearI8Plan p = moe::linear_w8a8_plan(s->rows, s->K, s->N, s->act);
  plan[0] = p.kernel;
  plan[1] = p.depth;
  plan[2] = s->x_dtype == MOE_INT8 ? 0 : p.makes_codes ? 1 : 2;
  return MOE_OK;
}

size_t moe_layer_w8a8_workspace(const moe_shape* s) {
  if (moe_api::check_shape(s, 16, 16)) return 0;
  return moe::layer_w8a8_workspace_bytes(s->T, s->H, s->I, s->E, s->k);
}

moe_status moe_layer_w8a8(const moe_shape* s, const float* logits, const void* x, int32_t x_dtype,
                          const int8_t* w13, const float* s13, const int8_t* w2, const float* s2,
                          const void* residual, int32_t* topk_ids, float* topk_w,
                          int32_t* expert_offsets, void* out, int32_t out_dtype, void* ws,
                          size_t ws_bytes, void* stream) {
  moe_status st = moe_api::check_shape(s, 16, 16);
  if (st) return st;
  if (x_dtype != MOE_BF16 && x_dtype != MOE_FP16)
    return fail(MOE_EINVAL, "x_dtype = %d is neither MOE_BF16 nor MOE_FP16", x_dtype);
  if (!floating(out_dtype))
    return fail(MOE_EINVAL, "out_dtype = %d is no MOE_BF16, MOE_FP16 or MOE_F32", out_dtype);
  if (s->T == 0 && !expert_offsets) return MOE_OK;
  if (expert_offsets) REQUIRE_PTR(expert_offsets);
  if (s->T > 0) {
    REQUIRE_PTR(logits);
    REQUIRE_PTR(x);
    REQUIRE_PTR(w13);
    REQUIRE_PTR(s13);
    REQUIRE_PTR(w2);
    REQUIRE_PTR(s2);
    if (residual) REQUIRE_PTR(residual);
    REQUIRE_PTR(topk_ids);
    REQUIRE_PTR(topk_w);
    REQUIRE_PTR(out);
  }
  const size_t need = moe::layer_w8a8_workspace_bytes(s->T, s->H, s->I, s->E, s->k);
  if (ws_bytes < need) return fail(MOE_EWORKSPACE, "layer workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE_PTR(ws);
  const int64_t T = s->T, H = s->H, I = s->I, E = s->E, k = s->k;
  const size_t out_bytes = values(T, H, out_dtype);
  if ((st = check_overlap({{"topk_ids", topk_ids, values(T, k, MOE_F32), true},
                           {"topk_w", topk_w, values(T, k, MOE_F32), true},
                           {"expert_offsets", expert_offsets, values(E + 1, 1, MOE_F32), true},
                           {"out", out, out_bytes, true},
                           {"ws", ws, need, true},
                           {"logits", logits, values(T, E, MOE_F32), false},
                           {"x", x, values(T, H, x_dtype), false},
                           {"w13", w13, values(E * 2 * I, H, MOE_INT8), false},
                           {"s13", s13, values(E * 2, I, MOE_F32), false},
                           {"w2", w2, values(E * H, I, MOE_INT8), false},
                           {"s2", s2, values(E, H, MOE_F32), false},
                           {"residual", residual == out ? nullptr : residual, out_bytes, false}})))
    return st;
  if ((st = check_device()) != MOE_OK) return st;
  const moe::LayerI8 l = {logits, x,  w13, s13, w2, s2, residual, topk_ids, topk_w, expert_offsets,
                          out, x_dtype, out_dtype, s->T, s->H, s->I, s->E, s->k};
  return launched(moe::launch_layer_w8a8(l, ws, static_cast<hipStream_t>(stream)),
                  "moe_layer_w8a8 launch");
}

moe_status moe_layer_w8a8_plan(const moe_shape* s, int32_t* plan) {
  const moe_status st = moe_api::check_shape(s, 16, 16);
  if (st) return st;
  if (!plan) return fail(MOE_EINVAL, "plan is NULL");
  const moe::LayerI8Plan p = moe::layer_w8a8_plan(s->T, s->H, s->I, s->E, s->k);
  plan[0] = p.way;
  plan[1] = p.up.take;
  plan[2] = p.up.makes_codes ? 1 : 2;
  plan[3] = p.down.take;
  plan[4] = p.down.makes_codes ? 1 : 2;
  return MOE_OK;
}

}  // extern "C"
