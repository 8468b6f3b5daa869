// step_api.hip -- the extern "C" entry points of moe_step.h: validate on the
// host, then launch on the caller's stream.
#include <math.h>

#include "step.h"

namespace {

inline moe_status_t dev(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EDEVICE; }
inline hipStream_t as_stream(moe_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

// A pointer to a zero-length array may be NULL; others are aligned to `a`.
inline bool bad(const void* p, int64_t n, uintptr_t a = 16)
{
    return n > 0 && (p == nullptr || (reinterpret_cast<uintptr_t>(p) & (a - 1)));
}
// An optional pointer: NULL, or aligned.
inline bool bad_opt(const void* p, uintptr_t a = 16)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}
// A gate's alignment: rows of gates are read as vectors, a token's one at a time.
inline uintptr_t gate_align(const moe_shape_t* s, int32_t gate_rows)
{
    return gate_rows > 0 ? 16 : s->dtype == MOE_BF16 ? 2 : 4;
}

moe_status_t check_blocks(int64_t rows, int64_t cols, int32_t dtype, const void* x, const void* q, const void* scales)
{
    if (rows < 0 || cols < 1 || (dtype != MOE_BF16 && dtype != MOE_F32)) return MOE_EINVAL;
    const int64_t lim = int64_t(1) << 40;
    if (cols >= lim || (rows > 0 && rows > (lim - 1) / cols)) return MOE_EINVAL;
    if (cols % moe::kMxBlock) return MOE_EUNSUPPORTED;
    return bad(x, rows) || bad(q, rows) || bad(scales, rows) ? MOE_EINVAL : MOE_OK;
}

moe_status_t check_mx(const moe_shape_t* s)
{
    const moe_status_t st = moe_check_shape(s);
    if (st != MOE_OK) return st;
    return s->dtype != MOE_BF16 || s->H % 128 || s->F % 128 ? MOE_EUNSUPPORTED : MOE_OK;
}

moe_status_t check_few(const moe_shape_t* s, int32_t form, int32_t shared_F)
{
    const moe_status_t st = moe_check_shape(s);
    if (st != MOE_OK) return st;
    if ((form != MOE_W_BF16 && form != MOE_W_MX8 && form != MOE_W_MX4) || shared_F < 0) return MOE_EINVAL;
    const int unit = moe::few_unit(form);
    if (s->dtype != MOE_BF16 || s->T > MOE_FEW_TOKENS || s->H > moe::kFewMaxH || s->H % unit || s->F % unit ||
        shared_F % unit)
        return MOE_EUNSUPPORTED;
    // (a projection's rows are addressed by 32-bit byte offsets)
    const int64_t wide = s->F > shared_F ? s->F : shared_F;
    return wide * s->H * 2 < (int64_t(1) << 32) - 128 ? MOE_OK : MOE_EUNSUPPORTED;
}
bool bad_weights(const moe_few_weights_t* w, int32_t form)
{
    return !w || bad(w->gate, 1) || bad(w->up, 1) || bad(w->down, 1) ||
           (form != MOE_W_BF16 && (bad(w->gate_scales, 1) || bad(w->up_scales, 1) || bad(w->down_scales, 1)));
}

}  // namespace

extern "C" {

moe_status_t moe_block_norm(const moe_shape_t* shape, const void* d_x, const void* d_residual, float alpha,
                            const void* d_w_post, const void* d_gate, int32_t gate_rows, const void* d_w_pre, float eps,
                            void* d_s, void* d_y, void* d_q, void* d_scales, float* d_rstd_post, float* d_rstd_pre,
                            moe_stream_t stream)
{
    const moe_status_t st = moe_check_shape(shape);
    if (st != MOE_OK) return st;
    if (!(eps > 0.0f) || !isfinite(eps) || !isfinite(alpha) || gate_rows < 0) return MOE_EINVAL;
    const int64_t T = shape->T;
    if (bad(d_x, T) || bad_opt(d_residual) || bad_opt(d_w_post) || bad_opt(d_gate, gate_align(shape, gate_rows)) ||
        bad_opt(d_w_pre) || bad_opt(d_s) || bad_opt(d_y) || bad_opt(d_q) || bad_opt(d_scales) ||
        bad_opt(d_rstd_post, 4) || bad_opt(d_rstd_pre, 4))
        return MOE_EINVAL;
    if (!d_w_post && d_rstd_post) return MOE_EINVAL;
    if (!d_w_pre && (d_y || d_q || d_scales || d_rstd_pre)) return MOE_EINVAL;
    if (T > 0 && !d_s && !d_y && !d_q && !d_rstd_post && !d_rstd_pre) return MOE_EINVAL;
    if ((d_q == nullptr) != (d_scales == nullptr)) return MOE_EINVAL;
    if (d_y && d_y == d_s) return MOE_EINVAL;
    if (d_q && shape->H % moe::kMxBlock) return MOE_EUNSUPPORTED;
    const MoeBlockNorm a{d_x, d_residual, alpha, d_w_post, d_gate, gate_rows, d_w_pre, eps, d_s, d_y, d_q, d_scales,
                         d_rstd_post, d_rstd_pre};
    return dev(moe_launch_block_norm(*shape, a, as_stream(stream)));
}

size_t moe_block_norm_backward_workspace_bytes(const moe_shape_t* shape, int32_t gate_rows)
{
    if (moe_check_shape(shape) != MOE_OK || gate_rows < 0) return 0;
    return moe::block_norm_bwd_ws(*shape, gate_rows);
}

moe_status_t moe_block_norm_backward(const moe_shape_t* shape, const void* d_x, const float* d_rstd_post,
                                     const void* d_s, const float* d_rstd_pre, float alpha, const void* d_w_post,
                                     const void* d_gate, int32_t gate_rows, const void* d_w_pre, const void* d_dy,
                                     const void* d_ds, void* d_dx, void* d_dresidual, float* d_dw_post, float* d_dgate,
                                     float* d_dw_pre, void* d_ws, size_t ws_bytes, moe_stream_t stream)
{
    const moe_status_t st = moe_check_shape(shape);
    if (st != MOE_OK) return st;
    if (!isfinite(alpha) || gate_rows < 0) return MOE_EINVAL;
    const int64_t T = shape->T;
    if (bad(d_x, T) || bad_opt(d_w_post) || bad_opt(d_gate, gate_align(shape, gate_rows)) || bad_opt(d_dy) ||
        bad_opt(d_ds) || bad(d_dx, T) || bad_opt(d_dresidual) || bad_opt(d_dw_post) || bad_opt(d_dw_pre) ||
        bad_opt(d_dgate, gate_rows > 0 ? 16 : 4) || bad(d_ws, 1))
        return MOE_EINVAL;
    if (T > 0 && !d_dy && !d_ds) return MOE_EINVAL;
    if (d_w_post ? bad(d_rstd_post, T, 4) : d_dw_post != nullptr) return MOE_EINVAL;
    if (d_dy ? bad(d_s, T) || bad(d_rstd_pre, T, 4) || bad(d_w_pre, 1) : T > 0 && d_dw_pre) return MOE_EINVAL;
    if (!d_gate && d_dgate) return MOE_EINVAL;
    if (T > 0 && d_dx == d_dresidual) return MOE_EINVAL;
    if (ws_bytes < moe::block_norm_bwd_ws(*shape, d_gate ? gate_rows : 0)) return MOE_EINVAL;
    const MoeBlockNormBwd a{d_x, d_rstd_post, d_s, d_rstd_pre, alpha, d_w_post, d_gate, gate_rows, d_w_pre, d_dy, d_ds,
                            d_dx, d_dresidual, d_dw_post, d_dgate, d_dw_pre};
    return dev(moe_launch_block_norm_backward(*shape, a, static_cast<float*>(d_ws), as_stream(stream)));
}

moe_status_t moe_mx4_quantize(int64_t rows, int64_t cols, int32_t dtype, const void* d_x, void* d_q, void* d_scales,
                              moe_stream_t stream)
{
    const moe_status_t st = check_blocks(rows, cols, dtype, d_x, d_q, d_scales);
    if (st != MOE_OK) return st;
    return dev(moe_launch_mx4_quantize(rows, cols, dtype, d_x, d_q, d_scales, as_stream(stream)));
}

moe_status_t moe_mx4_dequantize(int64_t rows, int64_t cols, int32_t dtype, const void* d_q, const void* d_scales,
                                void* d_x, moe_stream_t stream)
{
    const moe_status_t st = check_blocks(rows, cols, dtype, d_x, d_q, d_scales);
    if (st != MOE_OK) return st;
    return dev(moe_launch_mx4_dequantize(rows, cols, dtype, d_q, d_scales, d_x, as_stream(stream)));
}

size_t moe_mx4_workspace_bytes(const moe_shape_t* shape)
{
    return check_mx(shape) == MOE_OK ? moe::mx_ws_layout(*shape).total : 0;
}

moe_status_t moe_grouped_gemm_mx4(const moe_shape_t* shape, const void* d_a, const void* d_a_scales,
                                  const int32_t* d_plan, const void* d_w_gate, const void* d_gate_scales,
                                  const void* d_w_up, const void* d_up_scales, const void* d_w_down,
                                  const void* d_down_scales, void* d_y, void* d_ws, size_t ws_bytes, moe_stream_t stream)
{
    const moe_status_t st = check_mx(shape);
    if (st != MOE_OK) return st;
    const int64_t T = shape->T;
    if (bad(d_a, T) || bad(d_a_scales, T) || bad(d_plan, 1, 4) || bad(d_w_gate, 1) || bad(d_gate_scales, 1) ||
        bad(d_w_up, 1) || bad(d_up_scales, 1) || bad(d_w_down, 1) || bad(d_down_scales, 1) || bad(d_y, T) || bad(d_ws, 1))
        return MOE_EINVAL;
    if (ws_bytes < moe::mx_ws_layout(*shape).total) return MOE_EINVAL;
    const MoeMxWeights w{static_cast<const uint8_t*>(d_w_gate), static_cast<const uint8_t*>(d_gate_scales),
                         static_cast<const uint8_t*>(d_w_up), static_cast<const uint8_t*>(d_up_scales),
                         static_cast<const uint8_t*>(d_w_down), static_cast<const uint8_t*>(d_down_scales)};
    return dev(moe_launch_grouped_gemm_mx4(*shape, d_a, d_a_scales, d_plan, w, d_y, static_cast<char*>(d_ws),
                                           as_stream(stream)));
}

size_t moe_few_workspace_bytes(const moe_shape_t* shape, int32_t form, int32_t shared_F)
{
    if (check_few(shape, form, shared_F) != MOE_OK) return 0;
    return moe::few_ws_layout(*shape, shared_F).total;
}

moe_status_t moe_few_layer(const moe_shape_t* shape, int32_t form, const void* d_x, const void* d_w_router,
                           const float* d_bias, const moe_few_weights_t* h_routed, const moe_few_weights_t* h_shared,
                           int32_t shared_F, void* d_out, int32_t* d_ids, float* d_w, int32_t* d_err, void* d_ws,
                           size_t ws_bytes, moe_stream_t stream)
{
    const moe_status_t st = check_few(shape, form, shared_F);
    if (st != MOE_OK) return st;
    const int64_t T = shape->T;
    if (bad(d_x, T) || bad(d_w_router, 1) || bad_opt(d_bias, 4) || bad_weights(h_routed, form) || bad(d_out, T) ||
        bad_opt(d_ids, 4) || bad_opt(d_w, 4) || bad(d_err, 1, 4) || bad(d_ws, 1))
        return MOE_EINVAL;
    if ((h_shared != nullptr) != (shared_F > 0) || (h_shared && bad_weights(h_shared, form))) return MOE_EINVAL;
    if (ws_bytes < moe::few_ws_layout(*shape, shared_F).total) return MOE_EINVAL;
    const MoeFew a{d_x, d_w_router, d_bias, *h_routed, h_shared ? *h_shared : moe_few_weights_t{}, form, shared_F,
                   d_out, d_ids, d_w, d_err};
    return dev(moe_launch_few(*shape, a, static_cast<char*>(d_ws), as_stream(stream)));
}

}  // extern "C"
