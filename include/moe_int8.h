/*
 * moe_int8.h — C ABI of libmoe, third part: a block served in 8-bit integers on AMD
 * Instinct MI355X (gfx950), around and with the W8A8 experts of moe.h.
 *
 *   moe_quant_rows   token rows to int8 codes with a scale per token
 *   moe_linear_w8a8  y = act(x W^T + bias) + residual on int8 codes with scales per
 *                    token and per output channel (shared experts, projections)
 *   moe_layer_w8a8   the whole routed W8A8 layer in one call
 *
 * The conventions of moe.h hold for every call: device pointers to row-major
 * contiguous arrays, 16-byte aligned; arguments checked on the host before anything is
 * enqueued; no allocation, no synchronization, no pointer kept past the call; outputs
 * must not alias inputs (but a residual may be the output itself); calls on distinct
 * streams with distinct workspaces may run concurrently; two runs on the same inputs
 * give identical bits. A workspace holds nothing between calls.
 *
 * Codes of a row: s = max|x| / 127 in float32 (IEEE division), q = x / s to the nearest
 * whole number, ties to even, clamped to [-127, 127]; s = 0 and q = 0 for a row of zeros.
 * For rows of finite values that is the rule of moe_grouped_w8a8_ffn, which has none for
 * others; here a row that holds an infinity or a NaN gets s = NaN and q = 0: all that is
 * computed from it is NaN, and other rows are not touched.
 */
#ifndef MOE_INT8_H
#define MOE_INT8_H

#include "moe.h"
#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_INT8 3
#define MOE_INT8_MAX_K 65536   /* largest K: sums of its products fit 32 bits */

/*
 * moe_quant_rows — int8 codes and scales of rows.
 *   x      x_dtype (MOE_BF16, MOE_FP16 or MOE_F32) [rows, K]
 *   q      int8 [rows, K];  scale  float32 [rows]
 * Requires rows >= 0, K a positive multiple of 8, at most MOE_INT8_MAX_K.
 */
MOE_API moe_status moe_quant_rows(const void* x, int32_t x_dtype, int32_t rows, int32_t K,
                                  int8_t* q, float* scale, void* stream);

/*
 * Shape of an int8 product. Let No = N/2 for MOE_ACT_SWIGLU and N otherwise.
 *   rows     rows of y, at most 2^31 - 2^16; rows*max(N, K) <= 2^38
 *   K        a multiple of 16, at most MOE_INT8_MAX_K
 *   N        a multiple of 8 (of 16 for SWIGLU), at most 2^20; N*K <= 2^30
 *   x_dtype  MOE_INT8 (codes, with x_scale), MOE_BF16 or MOE_FP16 (values: the call
 *            makes their codes)
 *   y_dtype  MOE_BF16, MOE_FP16 or MOE_F32
 *   act      MOE_ACT_*
 */
typedef struct {
  int32_t rows;
  int32_t K;
  int32_t N;
  int32_t x_dtype;
  int32_t y_dtype;
  int32_t act;
} moe_w8_shape;

/*
 * moe_linear_w8a8 — a dense product of int8 codes with its epilogue.
 *   z[t, n] = (sum_k q[t, k] w[n, k]) * x_scale[t] * w_scale[n] + bias[n]
 *   y = act(z) + residual
 *   x         int8 [rows, K], or x_dtype [rows, K], whose codes (those of
 *             moe_quant_rows) the call makes
 *   x_scale   float32 [rows] with MOE_INT8, NULL otherwise
 *   w         int8 [N, K];  w_scale  float32 [N]
 *   bias      float32 [N] or NULL
 *   residual  y_dtype [rows, No] or NULL; may be y itself (added in place)
 *   y         y_dtype [rows, No]
 * The sum is exact in 32 bits for every value of the codes; it is rounded to float32
 * once and the rest is float32 with one rounding to y_dtype. `ws` must hold
 * moe_linear_w8a8_workspace(rows, K) bytes where x holds values; with codes it is not
 * used and may be NULL. The bytes grow with rows: a workspace for the most rows serves
 * fewer.
 */
MOE_API size_t moe_linear_w8a8_workspace(int32_t rows, int32_t K);
MOE_API moe_status moe_linear_w8a8(const moe_w8_shape* shape, const void* x, const float* x_scale,
                                   const int8_t* w, const float* w_scale, const float* bias,
                                   const void* residual, void* y, void* ws, size_t ws_bytes,
                                   void* stream);

/*
 * moe_linear_w8a8_plan — the kernel that a product of this shape runs on, chosen from the
 * shape alone. Host only; for tests and tuning: the numbers may change between versions.
 *   plan      int32 [3], written:
 *     [0]  0 to 7 as moe_product_plan's [0]; 8 weights through rings of the waves
 *     [1]  the depth of those rings, else 0
 *     [2]  the codes of x: 0 given, 1 made in the product's launch, 2 in one before it
 */
MOE_API moe_status moe_linear_w8a8_plan(const moe_w8_shape* shape, int32_t* plan);

/*
 * moe_layer_w8a8 — the whole W8A8 layer in one call: moe_route_topk's picks of
 * logits [T, E], the SwiGLU experts of moe_grouped_w8a8_ffn, and moe_combine's sum
 * added to a residual, by the definitions given there:
 *   out[t] = residual[t] + sum_{j < k} topk_w[t, j] * y[t, j],
 * summed in float32 in increasing j, the residual last, and rounded once to out_dtype.
 *   logits    float32 [T, E]
 *   x         x_dtype (MOE_BF16 or MOE_FP16) [T, H]
 *   w13       int8 [E, 2I, H] (rows [0, I) gate, [I, 2I) up);  s13  float32 [E, 2I]
 *   w2        int8 [E, H, I];  s2  float32 [E, H]
 *   residual  out_dtype [T, H] or NULL; may be out itself
 *   topk_ids  int32 [T, k];  topk_w  float32 [T, k]  (outputs)
 *   expert_offsets  int32 [E + 1] or NULL (output, as moe_permute's; feeds
 *             moe_expert_counts_accumulate)
 *   out       out_dtype (MOE_BF16, MOE_FP16 or MOE_F32) [T, H]
 * Requires what moe_grouped_w8a8_ffn does. `ws` must hold
 * moe_layer_w8a8_workspace(shape) bytes. Few tokens (up to 16 whose codes fit in LDS) take
 * two to four launches: two where T <= 8, T*H <= 16384 and T*k*I <= 16384; some tens take
 * five, more tokens seven to nine.
 * Which kernels run depends on the shape alone, and each result is the definition's, h
 * within its float32 roundings. Between kernels a code of h whose quotient lies next to
 * the middle of two whole numbers may be either of them: each such code moves the outputs
 * of its token by topk_w * s * w2 * s2, with s the scale of its row of h.
 */
MOE_API size_t moe_layer_w8a8_workspace(const moe_shape* shape);
MOE_API moe_status moe_layer_w8a8(const moe_shape* shape, const float* logits, const void* x,
                                  int32_t x_dtype, const int8_t* w13, const float* s13,
                                  const int8_t* w2, const float* s2, const void* residual,
                                  int32_t* topk_ids, float* topk_w, int32_t* expert_offsets,
                                  void* out, int32_t out_dtype, void* ws, size_t ws_bytes,
                                  void* stream);

/*
 * moe_layer_w8a8_plan — the kernels that a layer of this shape runs on, as
 * moe_linear_w8a8_plan.
 *   plan      int32 [5], written:
 *     [0]  0 weights through rings of the waves, codes of all rows in LDS; 1 codes through
 *          the rings too, in units of 16 rows of an expert; 2 grouped tiles; 3 the tiles
 *          of moe_grouped_w8a8_ffn
 *     [1]  gate/up: with 0 and 1 the depth of the rings, with 2 the tiles as
 *          moe_product_plan's [0], else 0;  [2] the codes: 1 made in the product's launch,
 *          2 in one before it
 *     [3], [4]  the same for down
 */
MOE_API moe_status moe_layer_w8a8_plan(const moe_shape* shape, int32_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* MOE_INT8_H */
