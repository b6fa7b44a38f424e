/*
 * moe_block.h — C ABI of libmoe, second part: the floating-point operators of
 * the block around and beside the quantized routed layer of moe.h, with their
 * gradients, for AMD Instinct MI355X (gfx950).
 *
 *   moe_grouped_mm      y = act(x W_e^T) for rows grouped by expert, with bf16
 *                       or fp16 expert weights (layers kept unquantized, or
 *                       trained), and its gradients
 *   moe_linear          y = act(x W^T + bias) + residual (shared experts, the
 *                       router in training), and its gradients
 *   moe_block_norm      r' = r + scale * gate * rms(y; w_post), h = rms(r'; w_pre)
 *                       (the norms after one block and before the next, fused
 *                       with the residual stream), and its gradients
 *   moe_combine_backward  the gradients of moe_combine and of moe_route_topk's
 *                       softmax over the picks
 *
 * The conventions of moe.h hold for every call: device pointers to row-major
 * contiguous arrays, 16-byte aligned; arguments checked on the host before
 * anything is enqueued; no allocation, no synchronization, no pointer kept past
 * the call; outputs must not alias inputs (one exception is named at
 * moe_linear); calls on distinct streams with distinct workspaces may run
 * concurrently; no float atomics, so two runs on the same inputs give identical
 * bits. A workspace holds nothing between calls.
 *
 * Types: `dtype` below is MOE_BF16 or MOE_FP16, the type of activations and
 * weights. Products of it are exact in float32 and are summed in float32; each
 * value is rounded once, where it is written. Infinities and NaN follow IEEE
 * arithmetic and stay in the rows and columns they belong to.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_BF16 0
#define MOE_FP16 1
#define MOE_F32 2

/* Activations of a product's output z. Every one but SWIGLU is element-wise.
 * SWIGLU takes z of width N (a multiple of 16) to N/2:
 * y_i = silu(z_i) * z_(N/2 + i), the W13 layout of moe.h. Float32 results are
 * within 18 * 2^-24 of the activation's value in its tails too (silu to z = -87, gelu
 * to -13, 0 below). At an infinite z the formulas' 0 * infinity is NaN: silu and gelu
 * of -infinity, their derivatives at both. */
#define MOE_ACT_NONE 0
#define MOE_ACT_RELU 1
#define MOE_ACT_SILU 2
#define MOE_ACT_GELU 3 /* 0.5 z (1 + erf(z / sqrt 2)) */
#define MOE_ACT_SWIGLU 4

/*
 * Shape of a product. Let No = N/2 for MOE_ACT_SWIGLU and N otherwise.
 *   rows    rows of y (grouped: the capacity R of the grouped arrays), at most
 *           2^31 - 2^16; rows*max(N, K) <= 2^38
 *   K, N    multiples of 8 (N of 16 for SWIGLU), N*K <= 2^30
 *   E       experts (1 .. MOE_MAX_EXPERTS); moe_linear* ignore it. Weight
 *           gradients: 256 rows x 256 columns of an expert's take 512 threads of
 *           a launch that holds fewer than 2^32 (E*N*K below 2^39 where N and K
 *           are multiples of 256); MOE_ESHAPE otherwise, before any launch
 *   x_rows  rows of x when sorted_slot is given (x_rows*K <= 2^30); otherwise
 *           x has `rows` rows and this is ignored
 *   topk    with sorted_slot: x's row for grouped row p is sorted_slot[p] / topk
 *   dtype   MOE_BF16 or MOE_FP16
 *   act     MOE_ACT_*
 */
typedef struct {
  int32_t rows;
  int32_t K;
  int32_t N;
  int32_t E;
  int32_t x_rows;
  int32_t topk;
  int32_t dtype;
  int32_t act;
} moe_mm_shape;

/*
 * moe_grouped_mm — products grouped by expert over ragged row blocks.
 * For p in [expert_offsets[e], expert_offsets[e+1]):
 *   z[p, :] = x[src(p), :] . W_e^T      y[p, :] = act(z[p, :])
 * with src(p) = sorted_slot[p] / topk, or p where sorted_slot is NULL.
 *   x              dtype [x_rows or rows, K]
 *   w              dtype [E, N, K]
 *   expert_offsets int32 [E+1], ascending, within [0, rows] (moe_permute's)
 *   sorted_slot    int32 [rows] or NULL (moe_permute's)
 *   z              dtype [rows, N] or NULL: kept for the gradients
 *   y              y_dtype (dtype or MOE_F32) [rows, No]
 * Rows of z and y outside [expert_offsets[0], expert_offsets[E]) are left as
 * they were. Offsets are clamped to [0, rows] and sources to [0, x_rows) on the
 * device: values outside the contract give wrong rows, never an access out of
 * bounds.
 */
MOE_API moe_status moe_grouped_mm(const moe_mm_shape* shape, const void* x, const void* w,
                                  const int32_t* expert_offsets, const int32_t* sorted_slot,
                                  void* z, void* y, int32_t y_dtype, void* stream);

/*
 * moe_grouped_mm_backward — the gradients of moe_grouped_mm.
 *   dz[p, :] = act'(z[p, :]) dy[p, :]   (dy itself for MOE_ACT_NONE)
 *   dx[p, :] = dz[p, :] . W_e           dw_e = sum over p of dz[p, :]^T x[src(p), :]
 *   dy  dtype [rows, No];  z  dtype [rows, N] (NULL only for MOE_ACT_NONE)
 *   w   dtype [E, N, K] (NULL if dx is);  x  as above (NULL if dw is)
 *   dx  dx_dtype (dtype or MOE_F32) [rows, K] or NULL, one row per grouped row
 *       (moe_combine with weights of one sums a token's picks); rows outside
 *       the experts' blocks are left as they were
 *   dw  dw_dtype (dtype or MOE_F32) [E, N, K] or NULL; every element is
 *       written (zero for an expert without rows)
 * dz is rounded to dtype where it enters the products (they run on dtype
 * operands); for MOE_ACT_NONE it is dy, unrounded. That rounding is one more of
 * dtype's half steps in dx and dw, and in MOE_FP16 it takes a dz under 2^-25 to zero
 * and one of 65520 or more to infinity, even where its factors (SwiGLU: dy, up and
 * silu') are in range: scale the loss for MOE_FP16, as for any gradient in that type.
 * `ws` must hold moe_grouped_mm_backward_workspace(shape) bytes (may be NULL when
 * that is 0).
 */
MOE_API size_t moe_grouped_mm_backward_workspace(const moe_mm_shape* shape);
MOE_API moe_status moe_grouped_mm_backward(const moe_mm_shape* shape, const void* dy,
                                           const void* x, const void* w, const void* z,
                                           const int32_t* expert_offsets,
                                           const int32_t* sorted_slot, void* dx, int32_t dx_dtype,
                                           void* dw, int32_t dw_dtype, void* ws, size_t ws_bytes,
                                           void* stream);

/*
 * moe_linear — a dense product with its epilogue.
 *   z = x . W^T + bias;   y = act(z) + residual
 *   x         dtype [rows, K];  w  dtype [N, K]
 *   bias      dtype [N] or NULL
 *   residual  y_dtype [rows, No] or NULL; may be y itself (added in place)
 *   z         dtype [rows, N] or NULL: kept for the gradients
 *   y         y_dtype (dtype or MOE_F32) [rows, No]
 */
MOE_API moe_status moe_linear(const moe_mm_shape* shape, const void* x, const void* w,
                              const void* bias, const void* residual, void* z, void* y,
                              int32_t y_dtype, void* stream);

/*
 * moe_linear_backward — the gradients of moe_linear.
 *   dz = act'(z) dy;  dx = dz . W;  dw = dz^T . x;  dbias = sum over rows of dz
 *   (the residual's gradient is dy)
 *   dy     dy_dtype (dtype or MOE_F32) [rows, No]
 *   z      dtype [rows, N] (NULL only for MOE_ACT_NONE)
 *   w      dtype [N, K] (NULL if dx is);  x  dtype [rows, K] (NULL if dw is)
 *   dx     dx_dtype (dtype or MOE_F32) [rows, K] or NULL
 *   dw     dw_dtype (dtype or MOE_F32) [N, K] or NULL
 *   dbias  dw_dtype [N] or NULL
 * dz is rounded to dtype where it enters the products (as in
 * moe_grouped_mm_backward: in MOE_FP16 a float32 dy does not widen its range), not
 * in dbias. With rows = 0, dw and dbias are set to zero. `ws` must hold
 * moe_linear_backward_workspace(shape) bytes, which grow with rows: a workspace
 * for the most rows serves fewer. They count a dz of rows * N values always: the
 * shape does not say whether dy itself is dz (MOE_ACT_NONE, dy of dtype).
 */
MOE_API size_t moe_linear_backward_workspace(const moe_mm_shape* shape);
MOE_API moe_status moe_linear_backward(const moe_mm_shape* shape, const void* dy,
                                       int32_t dy_dtype, const void* x, const void* w,
                                       const void* z, void* dx, int32_t dx_dtype, void* dw,
                                       void* dbias, int32_t dw_dtype, void* ws, size_t ws_bytes,
                                       void* stream);

/*
 * moe_product_plan — the kernels that a product of this shape and its gradients run
 * on, chosen by estimated time from the shape alone. Host only; for tests and tuning:
 * the numbers may change between versions.
 *   grouped   nonzero: moe_grouped_mm's, else moe_linear's
 *   plan      int32 [6], written:
 *     [0]  forward: 0 tiles of 256x256, 1 128x128, 2 64x128, 3 64x64, 4 128x256,
 *          5 128x128 of four stages, 6 and 7 rows by 16 and by 32
 *     [1]  gradients: 0 each in a launch of its own; both in one launch (where both
 *          are asked for) of 1 128x128 or 2 64x64 tiles
 *     [2]  dx's tiles in a launch of its own (numbers as in [0]);  [3] its parts
 *     [4]  dw's: 0 256x256, 1 256x128, 2 128x128, 3 64x64;  [5] its parts
 */
MOE_API moe_status moe_product_plan(const moe_mm_shape* shape, int32_t grouped, int32_t* plan);

/* How block_norm's gate broadcasts over y [T, H]. */
#define MOE_GATE_NONE 0
#define MOE_GATE_CHANNEL 1 /* gate [H]    */
#define MOE_GATE_TOKEN 2   /* gate [T]    */
#define MOE_GATE_ELEMENT 3 /* gate [T, H] */

#define MOE_NORM_MAX_H 16384

/*
 * Shape of a block norm.
 *   T        tokens (>= 0)
 *   H        width, a multiple of 8, at most MOE_NORM_MAX_H
 *   dtype    MOE_BF16 or MOE_FP16: h, the weights and the gate
 *   r_dtype  dtype or MOE_F32: the residual stream r, r_out
 *   y_dtype  dtype or MOE_F32: the block's output y (moe_combine's is float32)
 *   gate     MOE_GATE_*
 *   scale    factor of the block's contribution
 *   eps      added to the mean square (> 0)
 */
typedef struct {
  int32_t T;
  int32_t H;
  int32_t dtype;
  int32_t r_dtype;
  int32_t y_dtype;
  int32_t gate;
  float scale;
  float eps;
} moe_norm_shape;

/*
 * moe_block_norm — the norm after a block, its gated and scaled addition to the
 * residual stream, and the norm before the next block, in one pass:
 *   n     = y * w_post / sqrt(mean(y^2) + eps)      (n = y where w_post is NULL)
 *   r_out = r + scale * gate * n                    (r_out = r where y is NULL)
 *   h     = r_out * w_pre / sqrt(mean(r_out^2) + eps)
 * h is computed from r_out before it is rounded. The mean squares are float32: a row
 * whose squares sum to 2^128 or more (values of about 1e19) has an infinite one.
 *   y       y_dtype [T, H] or NULL (then w_post, gate and r_out must be NULL)
 *   r       r_dtype [T, H]
 *   r_out   r_dtype [T, H], written where y is given (may be NULL)
 *   h       dtype [T, H], with w_pre dtype [H]; both or neither
 *   w_post  dtype [H] or NULL;  gate dtype, NULL for MOE_GATE_NONE
 * At least one of r_out and h.
 */
MOE_API moe_status moe_block_norm(const moe_norm_shape* shape, const void* r, const void* y,
                                  const void* w_post, const void* gate, const void* w_pre,
                                  void* r_out, void* h, void* stream);

/*
 * moe_block_norm_backward — the gradients of moe_block_norm.
 *   r_out    r_dtype [T, H]: the forward's (r itself where y was NULL); needed
 *            with dh only
 *   dr_out   r_dtype [T, H] or NULL: the gradient that reaches r_out directly
 *   dh       dtype [T, H] or NULL, with w_pre
 *   y, w_post, gate  as in the forward
 *   dr       r_dtype [T, H]: dr_out + the gradient through h
 *   dy       y_dtype [T, H] or NULL (y given)
 *   dw_post, dw_pre  float32 [H] or NULL
 *   dgate    float32 [H] (CHANNEL), float32 [T] (TOKEN), dtype [T, H] (ELEMENT),
 *            or NULL
 * At least one of dr_out and dh. Sums over tokens run in a fixed order. `ws`
 * must hold moe_block_norm_backward_workspace(T, H) bytes (used for dw_post,
 * dw_pre and a CHANNEL gate's gradient; may be NULL where none is asked for).
 */
MOE_API size_t moe_block_norm_backward_workspace(int32_t T, int32_t H);
MOE_API moe_status moe_block_norm_backward(const moe_norm_shape* shape, const void* r_out,
                                           const void* dr_out, const void* dh, const void* y,
                                           const void* w_post, const void* gate,
                                           const void* w_pre, void* dr, void* dy, float* dw_post,
                                           float* dw_pre, void* dgate, void* ws, size_t ws_bytes,
                                           void* stream);

/*
 * moe_combine_backward — the gradients of out[t] = sum_j w[t, j] y[slot_pos[t*k + j]]
 * in the expert outputs and the router weights, and through the softmax over
 * the picks in the router logits.
 *   dy[slot_pos[t*k + j], :] = topk_w[t, j] * dout[t, :]
 *   dtopk_w[t, j] = sum_h dout[t, h] * y[slot_pos[t*k + j], h]
 *   dlogits[t, ids[t, j]] = topk_w[t, j] * (dtopk_w[t, j] - sum_i topk_w[t, i] dtopk_w[t, i])
 *                           and zero for the experts that t did not pick
 *   dout      float32 [T, H];  y  float32 [T*k, H] (NULL if dtopk_w and dlogits are)
 *   slot_pos  int32 [T*k] (moe_permute's; clamped to [0, T*k));  topk_w float32 [T, k]
 *   topk_ids  int32 [T, k] (needed with dlogits; ids outside [0, E) are dropped)
 *   dy        dy_dtype (MOE_BF16, MOE_FP16 or MOE_F32) [T*k, H] or NULL
 *   dtopk_w   float32 [T, k] or NULL;  dlogits float32 [T, E] or NULL
 * At least one output. Requires H % 8 == 0, 1 <= E <= MOE_MAX_EXPERTS,
 * 1 <= k <= min(E, MOE_MAX_TOPK).
 */
MOE_API moe_status moe_combine_backward(const float* dout, const float* y,
                                        const int32_t* slot_pos, const int32_t* topk_ids,
                                        const float* topk_w, int32_t T, int32_t H, int32_t E,
                                        int32_t k, void* dy, int32_t dy_dtype, float* dtopk_w,
                                        float* dlogits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
