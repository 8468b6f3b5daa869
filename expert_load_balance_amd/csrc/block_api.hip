// block_api.hip -- the extern "C" entry points of moe_block.h: validate on
// the host, then launch on the caller's stream.
#include <math.h>
#include <stdlib.h>

#include "mx.h"

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

moe_status_t check_mx(const moe_shape_t* s)
{
    const moe_status_t st = moe_check_shape(s);
    if (st != MOE_OK) return st;
    if (s->dtype != MOE_BF16 || s->H % 128 || s->F % 128) return MOE_EUNSUPPORTED;
    return MOE_OK;
}

inline int elem(int32_t dtype) { return dtype == MOE_BF16 ? 2 : 4; }

// pointers: the types and sources too (the size query's lists need not have any)
moe_status_t check_grads(int32_t n, const moe_grad_t* g, bool pointers, bool with_dst)
{
    if (n < 0 || (n > 0 && !g)) return MOE_EINVAL;
    for (int32_t i = 0; i < n; ++i) {
        if (g[i].count < 0 || g[i].count >= (int64_t(1) << 40)) return MOE_EINVAL;
        if (!pointers) continue;
        if (g[i].dtype != MOE_F32 && g[i].dtype != MOE_BF16) return MOE_EINVAL;
        if (bad(g[i].src, g[i].count, elem(g[i].dtype))) return MOE_EINVAL;
        if (with_dst && bad(g[i].dst, g[i].count, elem(g[i].dtype))) return MOE_EINVAL;
    }
    return MOE_OK;
}

struct Span {
    uintptr_t lo, hi;
    bool write;
};
int by_lo(const void* a, const void* b)
{
    const Span *x = static_cast<const Span*>(a), *y = static_cast<const Span*>(b);
    return x->lo < y->lo ? -1 : x->lo > y->lo ? 1 : 0;
}

// Whether some tensor's dst meets another's src or dst, or its own src in
// part: spans in address order; of those already passed, only the furthest end
// of a written one and of any one matter.
moe_status_t check_overlap(int32_t n, const moe_grad_t* g)
{
    if (n == 0) return MOE_OK;
    Span* sp = static_cast<Span*>(malloc(sizeof(Span) * 2 * (size_t)n));
    if (!sp) return MOE_EDEVICE;
    int m = 0;
    bool hit = false;
    for (int32_t i = 0; i < n && !hit; ++i) {
        if (g[i].count == 0) continue;
        const uintptr_t len = (uintptr_t)g[i].count * elem(g[i].dtype);
        const uintptr_t s = reinterpret_cast<uintptr_t>(g[i].src), d = reinterpret_cast<uintptr_t>(g[i].dst);
        sp[m++] = Span{d, d + len, true};
        if (s != d) {
            hit = s < d + len && d < s + len;
            sp[m++] = Span{s, s + len, false};
        }
    }
    if (!hit) {
        qsort(sp, (size_t)m, sizeof(Span), by_lo);
        uintptr_t end_any = 0, end_written = 0;
        for (int i = 0; i < m && !hit; ++i) {
            hit = sp[i].lo < end_written || (sp[i].write && sp[i].lo < end_any);
            if (sp[i].hi > end_any) end_any = sp[i].hi;
            if (sp[i].write && sp[i].hi > end_written) end_written = sp[i].hi;
        }
    }
    free(sp);
    return hit ? MOE_EINVAL : MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_rmsnorm(const moe_shape_t* shape, const void* d_x, const void* d_residual,
                         const void* d_weight, float eps, void* d_s, void* d_y, void* d_q,
                         void* d_scales, float* d_rstd, moe_stream_t stream)
{
    const moe_status_t st = moe_check_shape(shape);
    if (st != MOE_OK) return st;
    if (!(eps > 0.0f) || !isfinite(eps)) return MOE_EINVAL;
    const int64_t T = shape->T;
    if (bad(d_x, T) || bad_opt(d_residual) || bad(d_weight, 1) || bad_opt(d_s) || bad_opt(d_y) ||
        bad_opt(d_q) || bad_opt(d_scales) || bad_opt(d_rstd, 4))
        return MOE_EINVAL;
    if (T > 0 && !d_s && !d_y && !d_q && !d_rstd) return MOE_EINVAL;
    if ((d_q == nullptr) != (d_scales == nullptr)) return MOE_EINVAL;
    if (d_y && d_y == d_s) return MOE_EINVAL;
    if (d_q && shape->H % moe::kMxBlock) return MOE_EUNSUPPORTED;
    return dev(moe_launch_rmsnorm(*shape, d_x, d_residual, d_weight, eps, d_s, d_y, d_q, d_scales,
                                  d_rstd, as_stream(stream)));
}

size_t moe_rmsnorm_backward_workspace_bytes(const moe_shape_t* shape)
{
    if (moe_check_shape(shape) != MOE_OK) return 0;
    const int g = moe::norm_bwd_groups(*shape);
    return moe::align256((size_t)(g > 0 ? g : 1) * shape->H * 4);
}

moe_status_t moe_rmsnorm_backward(const moe_shape_t* shape, const void* d_s, const void* d_weight,
                                  const float* d_rstd, const void* d_dy, const void* d_ds,
                                  void* d_dx, float* d_dweight, void* d_ws, size_t ws_bytes,
                                  moe_stream_t stream)
{
    const moe_status_t st = moe_check_shape(shape);
    if (st != MOE_OK) return st;
    const int64_t T = shape->T;
    if (bad(d_s, T) || bad(d_weight, 1) || bad(d_rstd, T, 4) || bad(d_dy, T) || bad_opt(d_ds) ||
        bad(d_dx, T) || bad(d_dweight, 1) || bad(d_ws, 1))
        return MOE_EINVAL;
    if (ws_bytes < moe_rmsnorm_backward_workspace_bytes(shape)) return MOE_EINVAL;
    return dev(moe_launch_rmsnorm_backward(*shape, d_s, d_weight, d_rstd, d_dy, d_ds, d_dx,
                                           d_dweight, static_cast<float*>(d_ws), as_stream(stream)));
}

moe_status_t moe_mx_quantize(int64_t rows, int64_t cols, int32_t dtype, const void* d_x, void* d_q,
                             void* d_scales, moe_stream_t stream)
{
    if (rows < 0 || cols < 1 || (dtype != MOE_BF16 && dtype != MOE_F32)) return MOE_EINVAL;
    const int64_t lim = int64_t(1) << 40;
    if (cols >= lim || (rows > 0 && rows > (lim - 1) / cols)) return MOE_EINVAL;
    if (cols % moe::kMxBlock) return MOE_EUNSUPPORTED;
    if (bad(d_x, rows) || bad(d_q, rows) || bad(d_scales, rows)) return MOE_EINVAL;
    return dev(moe_launch_mx_quantize(rows, cols, dtype, d_x, d_q, d_scales, as_stream(stream)));
}

moe_status_t moe_permute_mx(const moe_shape_t* shape, const void* d_q, const void* d_scales,
                            const int32_t* d_ids, const int32_t* d_eidx, const int32_t* d_plan,
                            void* d_buf_q, void* d_buf_scales, int32_t* d_dest_row,
                            int32_t* d_row_src, moe_stream_t stream)
{
    const moe_status_t st = check_mx(shape);
    if (st != MOE_OK) return st;
    const int64_t T = shape->T;
    if (bad(d_q, T) || bad(d_scales, T) || bad(d_ids, T, 4) || bad(d_eidx, T, 4) ||
        bad(d_plan, 1, 4) || bad(d_buf_q, T) || bad(d_buf_scales, T) || bad(d_dest_row, T, 4) ||
        bad(d_row_src, T, 4))
        return MOE_EINVAL;
    return dev(moe_launch_permute_mx(*shape, d_q, d_scales, d_ids, d_eidx, d_plan, d_buf_q,
                                     d_buf_scales, d_dest_row, d_row_src, as_stream(stream)));
}

size_t moe_mx_workspace_bytes(const moe_shape_t* shape)
{
    if (check_mx(shape) != MOE_OK) return 0;
    return moe::mx_ws_layout(*shape).total;
}

moe_status_t moe_grouped_gemm_mx(const moe_shape_t* shape, const void* d_a, const void* d_a_scales,
                                 const int32_t* d_plan, const void* d_w_gate,
                                 const void* d_gate_scales, const void* d_w_up,
                                 const void* d_up_scales, const void* d_w_down,
                                 const void* d_down_scales, void* d_y, void* d_ws, size_t ws_bytes,
                                 moe_stream_t stream)
{
    const moe_status_t st = check_mx(shape);
    if (st != MOE_OK) return st;
    const int64_t T = shape->T;
    if (bad(d_a, T) || bad(d_a_scales, T) || bad(d_plan, 1, 4) || bad(d_w_gate, 1) ||
        bad(d_gate_scales, 1) || bad(d_w_up, 1) || bad(d_up_scales, 1) || bad(d_w_down, 1) ||
        bad(d_down_scales, 1) || bad(d_y, T) || bad(d_ws, 1))
        return MOE_EINVAL;
    if (ws_bytes < moe::mx_ws_layout(*shape).total) return MOE_EINVAL;
    const MoeMxWeights w{static_cast<const uint8_t*>(d_w_gate), static_cast<const uint8_t*>(d_gate_scales),
                         static_cast<const uint8_t*>(d_w_up), static_cast<const uint8_t*>(d_up_scales),
                         static_cast<const uint8_t*>(d_w_down), static_cast<const uint8_t*>(d_down_scales)};
    return dev(moe_launch_grouped_gemm_mx(*shape, d_a, d_a_scales, d_plan, w, d_y,
                                          static_cast<char*>(d_ws), as_stream(stream)));
}

size_t moe_grad_workspace_bytes(int32_t n, const moe_grad_t* h_grads)
{
    if (check_grads(n, h_grads, false, false) != MOE_OK) return 0;
    return moe_grad_ws_bytes(n, h_grads);
}

moe_status_t moe_grad_norm(int32_t n, const moe_grad_t* h_grads, float* d_norm, int32_t* d_err,
                           void* d_ws, size_t ws_bytes, moe_stream_t stream)
{
    const moe_status_t st = check_grads(n, h_grads, true, false);
    if (st != MOE_OK) return st;
    if (bad(d_norm, 1, 4) || bad(d_err, 1, 4) || bad(d_ws, 1, 8)) return MOE_EINVAL;
    if (ws_bytes < moe_grad_ws_bytes(n, h_grads)) return MOE_EINVAL;
    return dev(moe_launch_grad_norm(n, h_grads, d_norm, d_err, static_cast<double*>(d_ws),
                                    as_stream(stream)));
}

moe_status_t moe_grad_clip(int32_t n, const moe_grad_t* h_grads, float max_norm,
                           const float* d_norm, moe_stream_t stream)
{
    moe_status_t st = check_grads(n, h_grads, true, true);
    if (st != MOE_OK) return st;
    if (!(max_norm >= 0.0f) || !isfinite(max_norm) || bad(d_norm, 1, 4)) return MOE_EINVAL;
    st = check_overlap(n, h_grads);
    if (st != MOE_OK) return st;
    return dev(moe_launch_grad_clip(n, h_grads, max_norm, d_norm, as_stream(stream)));
}

}  // extern "C"
