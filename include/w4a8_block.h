/*
 * w4a8_block.h -- C ABI of the operators around the routed experts of a decoder
 * block, for AMD Instinct MI355X (gfx950): dense products with 8-bit integer
 * weights, the gated feed-forward block on such weights, and the norms before and
 * after a block.  Part of the same library as w4a8_moe.h, whose conventions (device
 * pointers, the caller's buffers and stream, status codes and
 * w4a8_moe_last_error, checks before any launch, results equal from run to run)
 * hold here too.
 *
 * The layers they serve: the per-channel form keeps attention projections, shared
 * experts and dense layers in 8-bit weights with 8-bit activations
 * ("GLM-5.3-Channel-INT4-w4a8" card, section 1: INT8 W8A8 next to the INT4 experts;
 * activations INT8, dynamic, per token).
 */
#ifndef W4A8_BLOCK_H
#define W4A8_BLOCK_H

#include "w4a8_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ---- Dense products with 8-bit integer weights --------------------------------
 * w4a8_moe_dense_i8 -- one weight matrix, a scale for each token and each channel:
 *     y[m, n] = a_scale[m] * w_scale[n] * sum_k a[m, k] * w[n, k] + bias[n] + add[m, n].
 *   The integer sum is exact (int32), then rounded to fp32 and multiplied by a_scale[m] and
 *   w_scale[n] in this order, each product rounded; bias and add are added in fp32 (a
 *   product and a sum may be one FMA), and y is rounded once more where it is bf16.
 *   a        : int8 [M][ld_a] (first K columns used), any codes in -128..127
 *              (w4a8_moe_quant_act_i8 and w4a8_moe_norm_quant_i8 write them); 16-byte
 *              aligned, ld_a % 16 == 0, K <= ld_a <= 2^22.   a_scale : fp32 [M].
 *   w        : int8 [N][K], 16-byte aligned.   w_scale : fp32 [N].  (Rows of bf16
 *              weights are quantized by w4a8_moe_quant_act_i8, which writes both.)
 *   bias     : fp32 [N] or NULL.
 *   add      : [M][N] of y's type or NULL; it may be y itself (y += ..), otherwise it
 *              must not overlap y.
 *   y        : [M][N], fp32 or bf16 (y_dtype W4A8_Y_F32 or W4A8_Y_BF16; rounded to
 *              nearest even), aligned to its elements; no overlap with a, w and the
 *              vectors (not checked).
 *   Rules    : M >= 0, 0 < N <= 2^24, 0 < K < 2^17, K % 16 == 0, M * N <= 2^40.
 *   Rows of a_scale that are not finite reach their own row of y only.
 */
int w4a8_moe_dense_i8(const int8_t* a, const float* a_scale, int64_t M, int64_t K, int64_t ld_a, const int8_t* w,
                      const float* w_scale, const float* bias, int64_t N, const void* add, void* y, int32_t y_dtype,
                      void* stream);

/*
 * w4a8_moe_mlp_i8 -- the gated feed-forward block on such weights (a shared expert, the
 * block of a dense layer):
 *     h[m, n]   = a_scale[m] * s13[n] * sum_k a[m, k] * w13[n, k];
 *     act[m, i] = silu(h[m, i]) * h[m, I + i], silu(z) = z / (1 + e^-z);
 *     sa[m]     = fl32(max_i |act[m, i]| / 127) (1.0 if that is 0),
 *     qa[m, i]  = the integer nearest to act[m, i] / sa[m], ties to even;
 *     y[m, n]   = sa[m] * s2[n] * sum_i qa[m, i] * w2[n, i] + add[m, n].
 *   Integer sums are exact; act is fp32 (hardware exponential and reciprocal: within a
 *   few ulp), so a code next to a border between two may fall on either side of it.
 *   a, a_scale : as in w4a8_moe_dense_i8 with K = H (16-byte rows: ld_a % 16 == 0).
 *   w13        : int8 [2I][H], gate rows 0..I-1, up rows I..2I-1.  s13 : fp32 [2I].
 *   w2         : int8 [H][I].  s2 : fp32 [H].  Both weights 16-byte aligned.
 *   add, y     : [M][H], as in w4a8_moe_dense_i8 (add may be y).
 *   workspace  : device memory of w4a8_moe_mlp_i8_workspace_bytes(M, H, I) bytes, 16-byte
 *                aligned; contents need no initialisation; calls that overlap must not
 *                share one.
 *   Rules      : M >= 0, 0 < H < 2^17, H % 16 == 0, 0 < I <= 65536, I % 128 == 0,
 *                M * max(H, 2I) <= 2^40.
 */
int64_t w4a8_moe_mlp_i8_workspace_bytes(int64_t M, int64_t H, int64_t I);
int w4a8_moe_mlp_i8(const int8_t* a, const float* a_scale, int64_t M, int64_t H, int64_t ld_a, const int8_t* w13,
                    const float* s13, const int8_t* w2, const float* s2, int64_t I, const void* add, void* y,
                    int32_t y_dtype, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * ---- Norms before and after a block -------------------------------------------
 * w4a8_moe_norm_quant (_i8) -- before a block: RMS norm of each row and its codes,
 *     n[t, :] = weight * x[t, :] / sqrt(mean(x[t, :]^2) + eps)   (fp32);
 *     xn[t, :] = n rounded to bf16 (the router's and the layer's input);
 *     scale and codes of n, as it is before that rounding: sx[t] = fl32(max |n| / 448)
 *     (_i8: / 127), 1.0 if that is 0; qx = E4M3 (_i8: the integer) nearest to 448 n / max |n|
 *     (127 n / max |n|), ties to even: to the exact quotient of weight * x, the norm's factor
 *     being in neither (one within 2^-42 of a tie counts as the tie; where n is below 2^-100, of
 *     the product to a multiple of fp32's smallest number); _i8: rowsum[t] = sum of qx[t, :].
 *   x       : [T][ld_x], fp32 or bf16 (x_dtype: W4A8_Y_F32, W4A8_Y_BF16), 16-byte aligned
 *             rows (ld_x % 8 == 0 in bf16, % 4 in fp32), ld_x >= H.
 *   weight  : fp32 [H], 16-byte aligned.
 *   xn      : bf16 [T][H], 16-byte aligned, or NULL.
 *   qx, sx  : u8 E4M3 (int8) [T][H], 8-byte aligned, and fp32 [T]; both or neither NULL
 *             (not both them and xn).   rowsum : int32 [T], or NULL.
 *   Rules   : T >= 0, 0 < H <= 32768, H % 8 == 0, 2^-100 <= eps < infinity (below, the
 *             squares of values that matter next to eps leave fp32's normal range).
 *   Squares are summed in fp32; rows whose sum overflows it are scaled first.  A row with
 *   a NaN or an infinity has outputs without meaning and a scale of NaN; the other rows
 *   are what they are without it.
 */
int w4a8_moe_norm_quant(const void* x, int32_t x_dtype, int64_t T, int64_t H, int64_t ld_x, const float* weight,
                        float eps, uint16_t* xn_bf16, uint8_t* qx, float* sx, void* stream);
int w4a8_moe_norm_quant_i8(const void* x, int32_t x_dtype, int64_t T, int64_t H, int64_t ld_x, const float* weight,
                           float eps, uint16_t* xn_bf16, int8_t* qx, float* sx, int32_t* rowsum, void* stream);

/*
 * w4a8_moe_residual_norm -- after a block whose result is y: norm, gates and residual,
 *     p[t, :]   = post_weight * y[t, :] / sqrt(mean(y[t, :]^2) + eps), or y[t, :] without
 *                 post_weight;
 *     out[t, :] = r_scale * r[t, :] + token_gate[t] * gate * p[t, :]  (fp32, then r's type).
 *   y       : [T][ld_y], fp32 or bf16 (y_dtype).   r : [T][ld_r], fp32 or bf16 (r_dtype).
 *             Rows 16-byte aligned, as x above.
 *   post_weight, gate : fp32 [H], 16-byte aligned, or NULL (no norm; a gate of 1).
 *   token_gate : fp32 [T] or NULL (1).
 *   out     : [T][ld_out] of r's type, rows as r's.  It may be r itself or y itself (same
 *             address, type and row distance); no other overlap (not checked).
 *   Rules   : as w4a8_moe_norm_quant; r_scale finite.
 *
 * w4a8_moe_residual_norm_quant (_i8) -- the same and the norm before the next block in
 *   one pass: xn, qx, sx (and rowsum) as w4a8_moe_norm_quant's of out with weight
 *   next_weight, taken of out before it is rounded to r's type.
 */
int w4a8_moe_residual_norm(const void* y, int32_t y_dtype, int64_t ld_y, const void* r, int32_t r_dtype, int64_t ld_r,
                           int64_t T, int64_t H, const float* post_weight, const float* gate, const float* token_gate,
                           float r_scale, float eps, void* out, int64_t ld_out, void* stream);
int w4a8_moe_residual_norm_quant(const void* y, int32_t y_dtype, int64_t ld_y, const void* r, int32_t r_dtype,
                                 int64_t ld_r, int64_t T, int64_t H, const float* post_weight, const float* gate,
                                 const float* token_gate, float r_scale, float eps, void* out, int64_t ld_out,
                                 const float* next_weight, uint16_t* xn_bf16, uint8_t* qx, float* sx, void* stream);
int w4a8_moe_residual_norm_quant_i8(const void* y, int32_t y_dtype, int64_t ld_y, const void* r, int32_t r_dtype,
                                    int64_t ld_r, int64_t T, int64_t H, const float* post_weight, const float* gate,
                                    const float* token_gate, float r_scale, float eps, void* out, int64_t ld_out,
                                    const float* next_weight, uint16_t* xn_bf16, int8_t* qx, float* sx,
                                    int32_t* rowsum, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_BLOCK_H */
