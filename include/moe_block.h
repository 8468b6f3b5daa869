/*
 * moe_block.h -- the operators around one MoE layer (moe.h), in the same
 * library, libmoe.so, under the same conventions:
 *   moe_rmsnorm, moe_rmsnorm_backward   the norm in front of the layer, with
 *                                       the residual's addition and an 8-bit
 *                                       output
 *   moe_mx_quantize, moe_permute_mx,    the routed experts on 8-bit rows and
 *   moe_grouped_gemm_mx                 8-bit weights (serving)
 *   moe_grad_norm, moe_grad_clip        the global norm of a list of
 *                                       gradients, and clipping to it
 *
 * 8-bit blocks ("mx"). 32 consecutive values of a row share one scale 2^e,
 * stored as the byte e + 127 (e8m0); the values are e4m3 codes (1 sign, 4
 * exponent, 3 mantissa bits, largest 448, no infinity). For values v of a
 * block, e is the smallest integer >= -127 with max|v| <= 448 * 2^e, so no
 * code saturates, and each code is v / 2^e rounded to nearest even. A block
 * holding an infinity or NaN gets the scale byte 255 (NaN) and NaN codes. A
 * matrix of `rows` x `cols` (cols % 32 == 0) is codes uint8[rows][cols] and
 * scales uint8[rows][cols / 32].
 *
 * Beyond moe.h's conventions: device pointers of activations, weights, codes
 * and scales are 16-byte aligned (MOE_EINVAL otherwise); outputs overlap
 * inputs only where a call says so.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Root-mean-square norm of T rows of width H (shape->T, H and dtype; the
 * other fields only have to be valid), with the residual's addition:
 *   s = x + residual, one fp32 add rounded to dtype (s = x without residual);
 *   rstd = 1 / sqrt(mean(s^2) + eps);  v = s * rstd * weight  (fp32);
 *   y = v rounded to dtype;  q, scales = v in 8-bit blocks (from the fp32
 *   values: one rounding, not y's and another).
 *   d_x, d_residual dtype[T][H] (d_residual may be NULL); d_weight dtype[H];
 *   eps > 0, finite; outputs, each may be NULL (not all of them): d_s, d_y
 *   dtype[T][H]; d_q uint8[T][H] and d_scales uint8[T][H/32] (both or
 *   neither; H % 32 == 0, MOE_EUNSUPPORTED otherwise); d_rstd float[T].
 * d_s may be d_x or d_residual, and d_y may be d_x or d_residual (not
 * both outputs the same array). A row holding an infinity or NaN gives NaN
 * or zero outputs in that row only. */
moe_status_t moe_rmsnorm(const moe_shape_t *shape, const void *d_x, const void *d_residual,
                         const void *d_weight, float eps, void *d_s, void *d_y, void *d_q,
                         void *d_scales, float *d_rstd, moe_stream_t stream);

/* Bytes of device workspace moe_rmsnorm_backward needs (per-workgroup sums of
 * the weight's gradient). 0 on a bad shape. */
size_t moe_rmsnorm_backward_workspace_bytes(const moe_shape_t *shape);

/* Backward of moe_rmsnorm through y. With xhat = s * rstd and g = dy * weight:
 *   dx = rstd * (g - xhat * mean(g * xhat)) + ds   (fp32, rounded once),
 *   dweight = sum over rows of dy * xhat           (fp32, overwritten; rows
 *   added in an order fixed by the shape).
 * dx is the gradient of x and of residual alike.
 *   d_s dtype[T][H] (moe_rmsnorm's s, or x where there was no residual);
 *   d_weight dtype[H]; d_rstd float[T] (moe_rmsnorm's); d_dy dtype[T][H];
 *   d_ds dtype[T][H] or NULL: the gradient that reaches s past the norm;
 *   d_dx dtype[T][H] out, may be d_dy or d_ds; d_dweight float[H] out;
 *   d_ws / ws_bytes >= moe_rmsnorm_backward_workspace_bytes(shape). */
moe_status_t moe_rmsnorm_backward(const moe_shape_t *shape, const void *d_s, const void *d_weight,
                                  const float *d_rstd, const void *d_dy, const void *d_ds,
                                  void *d_dx, float *d_dweight, void *d_ws, size_t ws_bytes,
                                  moe_stream_t stream);

/* A matrix in 8-bit blocks (weights once, when a model is loaded; rows that
 * no norm made). d_x dtype[rows][cols], dtype a moe_dtype_t; cols % 32 == 0
 * (MOE_EUNSUPPORTED otherwise); rows >= 0, cols >= 1, rows * cols < 2^40;
 * d_q uint8[rows][cols], d_scales uint8[rows][cols/32] out. */
moe_status_t moe_mx_quantize(int64_t rows, int64_t cols, int32_t dtype, const void *d_x,
                             void *d_q, void *d_scales, moe_stream_t stream);

/* moe_permute for 8-bit rows: token t's codes and scales go to its k rows of
 * the buffer. d_q uint8[T][H], d_scales uint8[T][H/32]; d_buf_q uint8[N][H],
 * d_buf_scales uint8[N][H/32] out; the other arguments, and every row's
 * place, as moe_permute. 8-bit shapes (this call and the next): dtype
 * MOE_BF16, H % 128 == 0 and F % 128 == 0 (MOE_EUNSUPPORTED otherwise). */
moe_status_t moe_permute_mx(const moe_shape_t *shape, const void *d_q, const void *d_scales,
                            const int32_t *d_ids, const int32_t *d_eidx, const int32_t *d_plan,
                            void *d_buf_q, void *d_buf_scales, int32_t *d_dest_row,
                            int32_t *d_row_src, moe_stream_t stream);

/* Bytes of device workspace moe_grouped_gemm_mx needs (tile schedule, row
 * map, the activations h in 8-bit blocks, fp32 partial tiles). 0 on a shape
 * that is bad or no 8-bit shape. Calls that may run at the same time, and
 * captured graphs that may, need a workspace each. */
size_t moe_mx_workspace_bytes(const moe_shape_t *shape);

/* moe_grouped_gemm on 8-bit blocks, with the scaled matrix instructions. For
 * row i of the buffer, held by expert e:
 *   g = W_gate[e] a_i, u = W_up[e] a_i (fp32 sums of scaled products);
 *   h = silu(g) * u in fp32, then in 8-bit blocks along F;
 *   y_i = W_down[e] h, rounded to bf16.
 * The matrix instructions align the products of 8 neighbouring values of K to
 * the largest and cut them at 2^-13 of its power of two (sums then carry about
 * 18 bits): where g and u come from such sums (experts of more than 64 rows), a
 * value of h next to the border of two codes may take either. Products and
 * values below 2^-126 may be taken as zero. So the bits of a row's y go by its
 * batch: by whether its expert has up to 64 rows there, and by the parts that the
 * launch cuts K into. Calls on the same inputs repeat theirs.
 *   d_a, d_a_scales uint8[N][H], uint8[N][H/32] (moe_permute_mx's buffer);
 *   d_w_gate, d_w_up uint8[E][F][H] with scales uint8[E][F][H/32];
 *   d_w_down uint8[E][H][F] with scales uint8[E][H][F/32]; d_plan from
 *   moe_plan; d_y bf16[N][H] out; d_ws / ws_bytes >=
 *   moe_mx_workspace_bytes(shape). Rows do not mix: a NaN stays in its row.
 * Serving only: the training path stays in bf16 (moe_grouped_gemm_train). */
moe_status_t moe_grouped_gemm_mx(const moe_shape_t *shape, const void *d_a, const void *d_a_scales,
                                 const int32_t *d_plan, const void *d_w_gate,
                                 const void *d_gate_scales, const void *d_w_up,
                                 const void *d_up_scales, const void *d_w_down,
                                 const void *d_down_scales, void *d_y, void *d_ws, size_t ws_bytes,
                                 moe_stream_t stream);

/* One gradient of a list. The list is host memory, read before the call
 * returns; tensors may be empty (src and dst then may be NULL). */
typedef struct moe_grad {
    const void *src; /* device dtype[count], aligned to its element size (one
                        off 16 bytes takes 1.2 to 6 times as long)            */
    void *dst;       /* moe_grad_clip: device dtype[count], may be src        */
    int64_t count;   /* elements, 0 <= count < 2^40                           */
    int32_t dtype;   /* moe_dtype_t                                           */
    int32_t reserved;/* 0                                                     */
} moe_grad_t;

/* Bytes of device workspace moe_grad_norm needs for this list (only n and the
 * counts are read). 0 when n < 0 or a count is out of range. */
size_t moe_grad_workspace_bytes(int32_t n, const moe_grad_t *h_grads);

/* norm = sqrt(sum of g^2 over every element of every tensor): the squares
 * are added in fp64, in an order fixed by the counts, and the root is rounded
 * to fp32. A tensor listed twice counts twice. n = 0 gives 0. When the norm
 * is infinite or NaN, *d_err |= MOE_ERR_NONFINITE.
 *   d_norm float[1] out; d_err int32[1] in/out; d_ws (8-byte aligned) /
 *   ws_bytes >= moe_grad_workspace_bytes(n, h_grads). */
moe_status_t moe_grad_norm(int32_t n, const moe_grad_t *h_grads, float *d_norm, int32_t *d_err,
                           void *d_ws, size_t ws_bytes, moe_stream_t stream);

/* dst = src * c for every tensor, c = max_norm / norm where norm > max_norm,
 * else 1 (the fp32 product, rounded to the tensor's type). A norm that is
 * infinite or NaN leaves the values as they are (c = 1): moe_grad_norm has
 * set the error word. Between the two calls a caller may combine the norm
 * with other ranks'. In place (dst == src) nothing is read or written when c
 * is 1. max_norm >= 0, finite; d_norm float[1], in. MOE_EINVAL when one
 * tensor's dst overlaps another's src or dst, or its own src in part. */
moe_status_t moe_grad_clip(int32_t n, const moe_grad_t *h_grads, float max_norm,
                           const float *d_norm, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
