// Host-side launchers of the block operators (moe_block.h). Arguments have been
// validated by block_api.cpp; each returns the launch status.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Launches of products. check: nothing is launched and no device is asked; returns
// hipErrorInvalidConfiguration where the launch would hold 2^32 threads or more.
struct MMArgs;
hipError_t launch_mm_nt(const MMArgs& a, int plan, bool fp16, hipStream_t s, bool check);
hipError_t launch_mm_nn(const MMArgs& a, int geom, bool fp16, hipStream_t s, bool check);
hipError_t launch_mm_tn(const MMArgs& a, int geom, bool fp16, hipStream_t s, bool check);
// The kernel of a forward product (launch_mm_nt's `plan`): 0 to 5 mm_pick_rows's
// geometries, 6 and 7 the few-row kernel with 16 and 32 rows a block. E 0: no experts.
int mm_forward_plan(int rows, int E, int N, int K, int act);
// out[n] = sum of part[parts][n] in order; out_type 0 bf16, 1 fp16, 2 float32.
// out NULL: none.
struct PartSum {
  const float* part;
  int parts, n;
  void* out;
  int out_type;
};
// How the gradients of a product are launched: both in one launch (pair 1 Mid,
// 2 Small) or apart (0), the geometries (mm_pick_rows's, mm_plan_tn's), the parts of
// each contraction. The same whichever gradients are asked for, so that one is the
// same bits alone and with the others.
struct MMBackwardPlan {
  int pair, nn, nn_splits, tn, tn_splits;
};
MMBackwardPlan mm_backward_plan(int rows, int E, int N, int K);   // E 0: no experts
// bytes for all parts of up to `rows` rows
size_t mm_backward_parts(int rows, int E, int N, int K);
// Both gradients, and a sum, in one launch.
hipError_t launch_mm_pair(const MMArgs& nn, const MMArgs& tn, const PartSum& sum, int pair,
                          bool fp16, hipStream_t s, bool check);

// dz = act'(z) dy. part NULL: rows [offsets[0], offsets[E]), or all where offsets is
// NULL. Otherwise all rows (offsets is not read), dz may be NULL, and part takes the
// column sums of dz over strips of rows, [dz_strips(rows, N, act)][N]; part_f32: their
// result is float32.
int dz_strips(int rows, int N, int act);
int dz_most_strips(int rows, int N, int act);   // of up to `rows` rows
hipError_t launch_dz(const void* dy, bool dy_f32, const void* z, const int* offsets, int E,
                     int rows, int N, int act, bool fp16, void* dz, float* part, bool part_f32,
                     hipStream_t s);
// out[e][i] = sum over the parts of part[e][s][i], in order; n values per e (a
// multiple of 4). out NULL: none.
struct SplitSum {
  const float* part;
  int splits, E;
  long long n;
  void* out;
  int out_type;
};
// All of these sums (those that there are) in one launch.
hipError_t launch_sums(const SplitSum& a, const SplitSum& b, const PartSum& c, hipStream_t s);

struct NormArgs {
  const void* r;        // forward: r; backward: r_out
  const void* y;
  const void* w_post;
  const void* gate;
  const void* w_pre;
  void* r_out;
  void* h;
  const void* dr_out;
  const void* dh;
  void* dr;
  void* dy;
  void* dgate;
  float* part;          // [blocks][2][H]: sums over tokens
  int T, H, gate_kind;
  int r_f32, y_f32;
  float scale, eps;
};
hipError_t launch_block_norm(const NormArgs& a, bool fp16, hipStream_t s);
int norm_backward_blocks(int T, int H);
hipError_t launch_block_norm_backward(const NormArgs& a, bool fp16, float* dw_pre, float* dw_post,
                                      float* dgate_channel, hipStream_t s);

struct LayerNormArgs {
  const void* r;        // forward: r; backward: r_out
  const void* y;
  const void* w;
  const void* b;
  void* r_out;
  void* h;
  const void* dr_out;
  const void* dh;
  void* dr;
  float* part;          // [blocks][2][H]: sums over tokens
  int T, H;
  int r_f32, y_f32;
  float eps;
};
hipError_t launch_layer_norm(const LayerNormArgs& a, bool fp16, hipStream_t s);
int layer_norm_backward_blocks(int T, int H);
hipError_t launch_layer_norm_backward(const LayerNormArgs& a, bool fp16, float* dw, float* db,
                                      hipStream_t s);

hipError_t launch_combine_backward(const float* dout, const float* y, const int* slot_pos,
                                   const int* ids, const float* w, int T, int H, int E, int k,
                                   void* dy, int dy_type, float* dw, float* dlogits,
                                   hipStream_t s);

}  // namespace moe
