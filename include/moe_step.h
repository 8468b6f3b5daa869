/*
 * moe_step.h -- one step through an MoE layer (moe.h) and between two of
 * them, in the same library, libmoe.so, under the conventions of moe.h and
 * moe_block.h:
 *   moe_block_norm, moe_block_norm_backward
 *                             what lies between two blocks of a residual
 *                             stream: the norm behind a block, its gate, the
 *                             residual's scale and addition, and the norm in
 *                             front of the next block
 *   moe_mx4_quantize, moe_mx4_dequantize, moe_grouped_gemm_mx4
 *                             weights in 4-bit blocks, and the routed experts
 *                             on them (serving)
 *   moe_few_layer             router to combine for a few tokens, on bf16,
 *                             8-bit or 4-bit weights
 *
 * 4-bit blocks ("mx4"). As the 8-bit blocks of moe_block.h, 32 consecutive
 * values of a row to a scale 2^e stored as the byte e + 127, with e2m1 codes
 * (1 sign, 2 exponent, 1 mantissa bit: 0, 1/2, 1, 3/2, 2, 3, 4, 6): e is the
 * smallest integer >= -127 with max|v| <= 6 * 2^e, so no code saturates, and
 * each code is v / 2^e rounded to nearest even. Code 2i of a row is the low
 * half of its byte i. e2m1 has no NaN: a block holding an infinity or NaN gets
 * the scale byte 255 (NaN) and codes of 0. A matrix of `rows` x `cols`
 * (cols % 32 == 0) is codes uint8[rows][cols / 2] and scales
 * uint8[rows][cols / 32].
 */
#ifndef MOE_STEP_H
#define MOE_STEP_H

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* T rows of width H (shape->T, H and dtype; the other fields only have to be
 * valid). x is a block's output, residual the stream that the block read:
 *   rstd_post = 1 / sqrt(mean(x^2) + eps);  n = x * rstd_post * w_post;
 *   s = alpha * residual + gate * n         (fp32, rounded once to dtype);
 *   rstd_pre = 1 / sqrt(mean(s^2) + eps);   v = s * rstd_pre * w_pre  (fp32);
 *   y = v rounded to dtype;  q, scales = v in 8-bit blocks (moe_block.h).
 *   d_x dtype[T][H]; d_residual dtype[T][H] or NULL (s = gate * n); alpha
 *   finite; d_w_post dtype[H] or NULL (n = x, then d_rstd_post is NULL);
 *   d_gate NULL (1) or, by gate_rows, 0: dtype[T], one value a token, and
 *   r >= 1: dtype[ceil(T / r)][H], row t / r for token t (1: a gate for every
 *   value; T or more: one for each channel); d_w_pre dtype[H] or NULL (no
 *   norm in front: d_y, d_q, d_scales and d_rstd_pre are NULL); eps > 0,
 *   finite; outputs, each may be NULL (not all of them): d_s, d_y dtype[T][H];
 *   d_q uint8[T][H] and d_scales uint8[T][H/32] (both or neither; H % 32 == 0,
 *   MOE_EUNSUPPORTED otherwise); d_rstd_post, d_rstd_pre float[T].
 * d_s may be d_x or d_residual, and d_y may be d_x or d_residual (not both
 * outputs the same array). An infinity or NaN stays in its row. */
moe_status_t moe_block_norm(const moe_shape_t *shape, const void *d_x, const void *d_residual,
                            float alpha, const void *d_w_post, const void *d_gate,
                            int32_t gate_rows, const void *d_w_pre, float eps, void *d_s, void *d_y,
                            void *d_q, void *d_scales, float *d_rstd_post, float *d_rstd_pre,
                            moe_stream_t stream);

/* Bytes of device workspace moe_block_norm_backward needs (sums of the
 * weights' and the gate's gradients over parts of the rows). 0 on a bad shape
 * or gate_rows < 0. Pass 0 where the gate has one value a token or is NULL. */
size_t moe_block_norm_backward_workspace_bytes(const moe_shape_t *shape, int32_t gate_rows);

/* Backward of moe_block_norm. With shat = s * rstd_pre, xhat = x * rstd_post:
 *   d = ds + rstd_pre * (dy * w_pre - shat * mean(dy * w_pre * shat));
 *   dresidual = alpha * d;  dgate = d * n, summed over what a gate multiplied;
 *   dn = gate * d;
 *   dx = rstd_post * (dn * w_post - xhat * mean(dn * w_post * xhat));
 *   dw_pre = sum over rows of dy * shat, dw_post of dn * xhat.
 * fp32 throughout, dx and dresidual rounded once; sums over rows are added in
 * an order fixed by the shape and gate_rows. dx's mean and a token's dgate are
 * differences of two sums, of what ds and dy give and of what the other mean takes
 * away: they are good to fp32's roundings of those sums' terms, not of d's.
 *   d_x, alpha, d_w_post, d_gate, gate_rows, d_w_pre as the forward's; d_s
 *   dtype[T][H], d_rstd_post, d_rstd_pre float[T] the forward's outputs;
 *   d_dy dtype[T][H] (the gradient of y) or NULL (none: d_w_pre, d_s,
 *   d_rstd_pre are not read, d_dw_pre is NULL); d_ds dtype[T][H] (the gradient
 *   that reaches s past the norm) or NULL; one of the two at least;
 *   d_w_post NULL: no norm behind (d_rstd_post is not read, d_dw_post NULL);
 *   outputs: d_dx dtype[T][H]; each may be NULL: d_dresidual dtype[T][H],
 *   d_dw_post, d_dw_pre float[H], d_dgate float, in d_gate's layout (NULL
 *   without a gate);
 *   d_ws / ws_bytes >= moe_block_norm_backward_workspace_bytes(shape,
 *   gate_rows), gate_rows 0 where d_gate is NULL.
 * d_dx and d_dresidual may be d_dy or d_ds (not both the same array). */
moe_status_t moe_block_norm_backward(const moe_shape_t *shape, const void *d_x,
                                     const float *d_rstd_post, const void *d_s,
                                     const float *d_rstd_pre, float alpha, const void *d_w_post,
                                     const void *d_gate, int32_t gate_rows, const void *d_w_pre,
                                     const void *d_dy, const void *d_ds, void *d_dx,
                                     void *d_dresidual, float *d_dw_post, float *d_dgate,
                                     float *d_dw_pre, void *d_ws, size_t ws_bytes,
                                     moe_stream_t stream);

/* A matrix in 4-bit blocks (weights once, when a model is loaded).
 *   d_x dtype[rows][cols], dtype a moe_dtype_t; cols % 32 == 0
 *   (MOE_EUNSUPPORTED otherwise); rows >= 0, cols >= 1, rows * cols < 2^40;
 *   d_q uint8[rows][cols/2], d_scales uint8[rows][cols/32] out. */
moe_status_t moe_mx4_quantize(int64_t rows, int64_t cols, int32_t dtype, const void *d_x,
                              void *d_q, void *d_scales, moe_stream_t stream);

/* The values of 4-bit blocks, code * 2^e rounded to dtype (bf16 holds every
 * value of magnitude 2^-126 and more exactly; below, bf16's subnormals round; 2^128
 * and more, the largest codes of scales of 2^126 and 2^127, are infinite). A scale
 * byte of 255 gives NaN.
 *   d_q uint8[rows][cols/2], d_scales uint8[rows][cols/32]; d_x
 *   dtype[rows][cols] out; limits as moe_mx4_quantize. */
moe_status_t moe_mx4_dequantize(int64_t rows, int64_t cols, int32_t dtype, const void *d_q,
                                const void *d_scales, void *d_x, moe_stream_t stream);

/* Bytes of device workspace moe_grouped_gemm_mx4 needs. 0 on a shape that is
 * bad or no 8-bit shape (moe_permute_mx). Calls that may run at the same time,
 * and captured graphs that may, need a workspace each. */
size_t moe_mx4_workspace_bytes(const moe_shape_t *shape);

/* moe_grouped_gemm_mx with weights in 4-bit blocks: rows and h stay in 8-bit
 * blocks, the products are the scaled matrix instructions' of 4-bit by 8-bit
 * codes, with their precision as described there; but gate and up of experts of up
 * to 64 rows are multiplied in two parts of the rows' codes, which the cut leaves
 * whole but for their last bits, where 8-bit weights take bf16 products. y is
 * rounded to bf16 before the combine, as there.
 *   d_a, d_a_scales uint8[N][H], uint8[N][H/32] (moe_permute_mx's buffer);
 *   d_w_gate, d_w_up uint8[E][F][H/2] with scales uint8[E][F][H/32];
 *   d_w_down uint8[E][H][F/2] with scales uint8[E][H][F/32]; d_plan from
 *   moe_plan; d_y bf16[N][H] out; d_ws / ws_bytes >=
 *   moe_mx4_workspace_bytes(shape). Rows do not mix: a NaN stays in its row. */
moe_status_t moe_grouped_gemm_mx4(const moe_shape_t *shape, const void *d_a, const void *d_a_scales,
                                  const int32_t *d_plan, const void *d_w_gate,
                                  const void *d_gate_scales, const void *d_w_up,
                                  const void *d_up_scales, const void *d_w_down,
                                  const void *d_down_scales, void *d_y, void *d_ws, size_t ws_bytes,
                                  moe_stream_t stream);

/* Weights of moe_few_layer's experts. MOE_W_BF16: bf16, no scales. MOE_W_MX8,
 * MOE_W_MX4: codes and scales of 8-bit or 4-bit blocks. */
typedef enum { MOE_W_BF16 = 0, MOE_W_MX8 = 1, MOE_W_MX4 = 2 } moe_weight_form_t;
typedef struct moe_few_weights {
    const void *gate, *up, *down;                      /* [E][F][H], [E][F][H], [E][H][F] */
    const void *gate_scales, *up_scales, *down_scales; /* of blocks; else not read        */
} moe_few_weights_t;

/* Most tokens of moe_few_layer. */
#define MOE_FEW_TOKENS 32

/* Bytes of device workspace moe_few_layer needs (scores, the choice,
 * the activations h, partial sums). shared_F: width of the shared expert, 0 without one. 0 on a
 * shape that moe_few_layer refuses. Calls that may run at the same time, and
 * captured graphs that may, need a workspace each. */
size_t moe_few_workspace_bytes(const moe_shape_t *shape, int32_t form, int32_t shared_F);

/* The whole layer for T <= MOE_FEW_TOKENS tokens:
 *   logits = x W_r^T; ids and gate weights w from them as moe_route;
 *   out[t] = sum_j w[t][j] * W_down[e] (silu(W_gate[e] x_t) * (W_up[e] x_t)),
 *            e = ids[t][j], in j order of sums in fp32
 *            (+ the same of the shared expert, weight 1), rounded once to bf16.
 * Products are of bf16 values with fp32 sums; h keeps 16 bits of its value (two
 * bf16), so that bf16's rounding of out is the only one that counts. Blocks widen
 * to bf16: exactly, with scales of 2^-124 to 2^119 (8-bit codes) and up to 2^125
 * (4-bit codes); beyond, values that bf16 does not hold round to it or are infinite.
 * Products and sums below 2^-126 may be taken as zero. Each live expert's weights
 * are read once for up to 16 of its tokens, and once for all of them where experts
 * have more than 8 on average (gate and up: if H <= 4096). No plan, no dispatch: R
 * and S of the shape are not used. The calls on 8-bit rows (moe_permute_mx and
 * moe_grouped_gemm_mx or _mx4) are about as fast on 8-bit weights where more than 16
 * tokens choose, and an expert has more than 12 of them on average (T * k / E); on
 * 4-bit weights they then take from a tenth more to a fifth less (32 tokens, every
 * expert chosen by all). With fewer they are slower.
 *   shape: dtype MOE_BF16; form a moe_weight_form_t, for the routed and the
 *   shared experts; MOE_W_MX8 and MOE_W_MX4 need H, F and shared_F multiples
 *   of 128, MOE_W_BF16 of 64; H <= 8192; H * F and H * shared_F below 2^31 - 64;
 *   else, and for more tokens or another dtype, MOE_EUNSUPPORTED;
 *   d_x bf16[T][H]; d_w_router bf16[E][H]; d_bias float[E] or NULL; h_routed:
 *   host memory, read before the call returns; h_shared with one expert of
 *   width shared_F, or NULL with shared_F 0; d_out bf16[T][H]; d_ids
 *   int32[T][k] and d_w float[T][k], the router's choice, each may be NULL;
 *   d_err int32[1] in/out (MOE_ERR_NONFINITE: a logit or bias is infinite or
 *   NaN); d_ws / ws_bytes >= moe_few_workspace_bytes(shape, form, shared_F).
 * d_out overlaps no input. Calls on the same inputs repeat their bits. */
moe_status_t moe_few_layer(const moe_shape_t *shape, int32_t form, const void *d_x,
                           const void *d_w_router, const float *d_bias,
                           const moe_few_weights_t *h_routed, const moe_few_weights_t *h_shared,
                           int32_t shared_F, void *d_out, int32_t *d_ids, float *d_w,
                           int32_t *d_err, void *d_ws, size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_STEP_H */
