// Host-side launchers of the int8 operators (moe_int8.h). Arguments have been
// validated by int8_api.cpp; each returns the launch status.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Types: 0 bf16, 1 fp16, 2 float32.
hipError_t launch_quant_rows(const void* x, int x_type, int rows, int K, int8_t* q, float* scale,
                             hipStream_t s);

struct LinearI8 {
  const int8_t* q;        // [rows, K]
  const float* q_scale;   // [rows]
  const int8_t* w;        // [N, K]
  const float* w_scale;   // [N]
  const float* bias;      // [N] or NULL
  const void* residual;   // like y, or NULL
  void* y;
  int y_type;
  int rows, K, N, act;
};
// The kernel of a product: mm_forward_plan's numbers, or kPlanRings (linear_few.h) with the
// depth of its rings. makes_codes: of values, whose codes the product's launch makes.
constexpr int kPlanRings = 8;
struct LinearI8Plan {
  int kernel, depth;
  bool makes_codes;
};
LinearI8Plan linear_w8a8_plan(int rows, int K, int N, int act);
// check: nothing is launched; hipErrorInvalidConfiguration where the launch would hold
// 2^32 threads or more.
hipError_t launch_linear_w8a8(const LinearI8& l, const LinearI8Plan& plan, hipStream_t s, bool check);
// Values (x_type 0 or 1) of a plan that makes their codes (q and q_scale are not read).
hipError_t launch_linear_w8a8_values(const LinearI8& l, const void* x, int x_type, hipStream_t s);

// out[p] = (q[src(p)] . W_e^T) scaled, float32, for the rows p of each expert e; src(p) =
// slot[p] / topk, or p where slot is NULL. swiglu: N is 2 I, out [rows, I].
struct GroupedI8 {
  const int8_t* q;        // [q_rows, K]
  const float* q_scale;   // [q_rows]
  const int8_t* w;        // [E, N, K]
  const float* w_scale;   // [E, N]
  const int* offsets;     // [E + 1]
  const int* slot;        // [rows] or NULL
  float* out;
  int rows, q_rows, topk, E, K, N;
  bool swiglu;
};
hipError_t launch_grouped_i8(const GroupedI8& g, hipStream_t s);

struct LayerI8 {
  const float* logits;
  const void* x;
  const int8_t* w13;
  const float* s13;
  const int8_t* w2;
  const float* s2;
  const void* residual;   // like out, or NULL
  int* ids;
  float* w;
  int* offsets;           // [E + 1] or NULL
  void* out;
  int x_type, out_type;   // x: 0 or 1
  int T, H, I, E, k;
};
// The kernels of a layer: a way, and for each of its products what it takes there.
enum LayerWay { kWayRings, kWayRingsByRows, kWayTiles, kWayLargeTiles };
struct LayerI8Half {
  int take;           // the depth of its rings; kWayTiles: mm_forward_plan's number
  bool makes_codes;   // codes made in the product's launch
};
struct LayerI8Plan {
  LayerWay way;
  LayerI8Half up, down;
};
LayerI8Plan layer_w8a8_plan(int T, int H, int I, int E, int k);
size_t layer_w8a8_workspace_bytes(int T, int H, int I, int E, int k);
hipError_t launch_layer_w8a8(const LayerI8& l, void* ws, hipStream_t s);

}  // namespace moe
