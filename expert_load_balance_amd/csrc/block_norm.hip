// block_norm.hip -- what lies between two blocks of a residual stream, and its
// backward:
//
//   rstd_post = (mean x^2 + eps)^-1/2, n = x rstd_post w_post,
//   s = round(alpha residual + gate n),
//   rstd_pre = (mean s^2 + eps)^-1/2, v = s rstd_pre w_pre,
//   y = round(v), (q, scales) = blocks(v).
//
// Bound by memory: each input is read once and each output written once. One
// workgroup takes one row and keeps it in registers over both norms' sums, as
// CH 16-byte vectors of x and of the residual per thread.
#include "rows.h"
#include "step.h"

namespace {

using moe::rows::rstd_of;
using moe::rows::store_mx;
using moe::rows::Vec;
using moe::rows::wg_sum;

constexpr int kMaxThreads = 1024;
constexpr int kMaxRows = 1 << 21;  // workgroups of a launch (2^32 threads at most)
constexpr int kRedCols = 64;       // columns per workgroup of the gradients' sum

// The arguments as the kernels take them: vectors of 16 bytes.
struct Fwd {
    int H, vecs;
    int64_t row0;                // of the launch
    const uint4 *x, *residual;
    float alpha, eps;
    const uint4 *w_post, *w_pre;
    const void* gate;
    uint32_t gate_rows;          // 0: a value a token
    uint4 *s, *y;
    uint8_t *q, *scales;
    float *rstd_post, *rstd_pre;
};

// The gate of a token as one value, or 1.
template <bool BF16>
__device__ __forceinline__ float token_gate(const void* gate, uint32_t gate_rows, int64_t row)
{
    if (!gate || gate_rows > 0) return 1.0f;
    return BF16 ? moe::bf16_bits_to_f32(static_cast<const uint16_t*>(gate)[row]) : static_cast<const float*>(gate)[row];
}
// Its row of gates, or null.
__device__ __forceinline__ const uint4* gate_row(const void* gate, uint32_t gate_rows, int64_t row, int vecs)
{
    return gate && gate_rows > 0 ? static_cast<const uint4*>(gate) + (int64_t)((uint32_t)row / gate_rows) * vecs : nullptr;
}

// s of one vector, rounded to the type (u: its bits, f: its values): x is f on
// entry, times the rstd already.
template <bool BF16>
__device__ __forceinline__ void step_of(float* f, uint4& u, const uint4& w, bool has_w, const uint4& g, bool has_g,
                                        float tg, const uint4& r, bool has_r, float alpha)
{
    using V = Vec<BF16>;
    float a[V::kN];
    if (has_w) {
        V::load(w, a);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[k] *= a[k];
    }
    if (has_g) {
        V::load(g, a);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[k] *= a[k];
    } else {
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[k] *= tg;
    }
    if (has_r) {
        V::load(r, a);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[k] = fmaf(alpha, a[k], f[k]);
    }
    u = V::store(f);
    V::load(u, f);
}

template <int N>
__device__ __forceinline__ double square_sum(const float* f, double ss)
{
#pragma unroll
    for (int k = 0; k < N; ++k) ss = fma((double)f[k], (double)f[k], ss);
    return ss;
}

// s, y may be x or residual: a thread stores a vector only after it read it
template <bool BF16, int CH, bool STREAM>
__global__ __launch_bounds__(kMaxThreads) void block_norm_kernel(const Fwd a)
{
    using V = Vec<BF16>;
    __shared__ double red[2][16];
    const int64_t row = a.row0 + blockIdx.x, base = row * a.vecs;
    const float tg = token_gate<BF16>(a.gate, a.gate_rows, row);
    const uint4* gr = gate_row(a.gate, a.gate_rows, row, a.vecs);
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 u[CH], r[CH], w1[CH], g[CH], w2[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        u[i] = r[i] = w1[i] = g[i] = w2[i] = none;
        if (c < a.vecs) {
            u[i] = moe::load16<STREAM>(a.x + base + c);
            if (a.residual) r[i] = moe::load16<STREAM>(a.residual + base + c);
            if (a.w_post) w1[i] = a.w_post[c];
            if (gr) g[i] = gr[c];
            if (a.w_pre) w2[i] = a.w_pre[c];
        }
    }
    float f[CH][V::kN], rs1 = 1.0f;
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < CH; ++i) V::load(u[i], f[i]);
    if (a.w_post) {
#pragma unroll
        for (int i = 0; i < CH; ++i) ss = square_sum<V::kN>(f[i], ss);
        rs1 = rstd_of(wg_sum(ss, red[0]), a.H, a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = rs1;
        ss = 0.0;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[i][k] *= rs1;
        step_of<BF16>(f[i], u[i], w1[i], a.w_post, g[i], gr, tg, r[i], a.residual, a.alpha);
        if (a.s && c < a.vecs) moe::store16<STREAM>(a.s + base + c, u[i]);
        ss = c < a.vecs ? square_sum<V::kN>(f[i], ss) : ss;
    }
    if (!a.w_pre) return;
    const float rs2 = rstd_of(wg_sum(ss, red[1]), a.H, a.eps);
    if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[row] = rs2;
    if (!a.y && !a.q) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        float w[V::kN];
        V::load(w2[i], w);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[i][k] = f[i][k] * rs2 * w[k];
        if (a.y && c < a.vecs) moe::store16<STREAM>(a.y + base + c, V::store(f[i]));
        if (a.q) store_mx<BF16>(f[i], base + c, c < a.vecs, a.q, a.scales);
    }
}

// Rows too wide for the registers: three passes over the row. s, where it is
// kept, may have replaced x or residual: it is read back then.
template <bool BF16>
__global__ __launch_bounds__(kMaxThreads) void block_norm_wide_kernel(const Fwd a)
{
    using V = Vec<BF16>;
    __shared__ double red[2][16];
    const int64_t row = a.row0 + blockIdx.x, base = row * a.vecs;
    const float tg = token_gate<BF16>(a.gate, a.gate_rows, row);
    const uint4* gr = gate_row(a.gate, a.gate_rows, row, a.vecs);
    const uint4 none = make_uint4(0, 0, 0, 0);
    float f[V::kN], rs1 = 1.0f;
    double ss = 0.0;
    if (a.w_post) {
        for (int c = threadIdx.x; c < a.vecs; c += blockDim.x) {
            V::load(a.x[base + c], f);
            ss = square_sum<V::kN>(f, ss);
        }
        rs1 = rstd_of(wg_sum(ss, red[0]), a.H, a.eps);
        if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = rs1;
    }
    auto step_at = [&](int c, uint4& u) {
        V::load(a.x[base + c], f);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[k] *= rs1;
        step_of<BF16>(f, u, a.w_post ? a.w_post[c] : none, a.w_post, gr ? gr[c] : none, gr, tg,
                      a.residual ? a.residual[base + c] : none, a.residual, a.alpha);
    };
    ss = 0.0;
    for (int c = threadIdx.x; c < a.vecs; c += blockDim.x) {
        uint4 u;
        step_at(c, u);
        if (a.s) a.s[base + c] = u;
        ss = square_sum<V::kN>(f, ss);
    }
    if (!a.w_pre) return;
    const float rs2 = rstd_of(wg_sum(ss, red[1]), a.H, a.eps);
    if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[row] = rs2;
    if (!a.y && !a.q) return;
    for (int c0 = 0; c0 < a.vecs; c0 += blockDim.x) {
        const int c = c0 + threadIdx.x;
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[k] = 0.0f;
        if (c < a.vecs) {
            float w[V::kN];
            uint4 u;
            if (a.s) V::load(a.s[base + c], f);
            else step_at(c, u);
            V::load(a.w_pre[c], w);
#pragma unroll
            for (int k = 0; k < V::kN; ++k) f[k] = f[k] * rs2 * w[k];
            if (a.y) a.y[base + c] = V::store(f);
        }
        if (a.q) store_mx<BF16>(f, base + c, c < a.vecs, a.q, a.scales);
    }
}

// ---------------------------------------------------------------- backward --
//   d = ds + rstd_pre (g - shat mean(g shat)), g = dy w_pre, shat = s rstd_pre;
//   dresidual = alpha d, dn = gate d,
//   dx = rstd_post (e - xhat mean(e xhat)), e = dn w_post, xhat = x rstd_post.
// A workgroup takes parts (runs of rows under one row of gates) b, b + G, ...
// and keeps the fp32 sums of dw_pre and dw_post of its columns over all of its
// rows, and those of dgate over a part, so that the sums' order is fixed.
struct Bwd {
    int H, vecs;
    int64_t T;
    moe::BlockNormParts p;
    const uint4 *x, *s, *w_post, *w_pre, *dy, *ds;
    const float *rstd_post, *rstd_pre;
    float alpha;
    const void* gate;
    uint32_t gate_rows;
    uint4 *dx, *dresidual;
    float *token_dgate;                     // a value a token
    float *part_post, *part_pre, *part_gate; // [G][H], [G][H], [parts][H], or null
};

template <int N>
__device__ __forceinline__ void store_sums(float* to, const float* v)
{
#pragma unroll
    for (int k = 0; k < N; k += 4)
        *reinterpret_cast<float4*>(to + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
}

template <bool BF16, int CH, int TH, bool STREAM>
__global__ __launch_bounds__(TH) void block_norm_bwd_kernel(const Bwd a)
{
    using V = Vec<BF16>;
    constexpr int N = V::kN;
    __shared__ float red[2][2][16];
    const float inv_h = 1.0f / (float)a.H;
    const uint4 none = make_uint4(0, 0, 0, 0);
    float acc_post[CH][N], acc_pre[CH][N], acc_gate[CH][N];
    uint4 w1[CH], w2[CH], gv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        w1[i] = c < a.vecs && a.w_post ? a.w_post[c] : none;
        w2[i] = c < a.vecs && a.w_pre ? a.w_pre[c] : none;
#pragma unroll
        for (int k = 0; k < N; ++k) acc_post[i][k] = acc_pre[i][k] = acc_gate[i][k] = 0.0f;
    }
    int turn = 0;
    for (int64_t part = blockIdx.x; part < a.p.parts; part += gridDim.x) {
        const int64_t group = part / a.p.per_group, r0 = group * a.p.group_rows + part % a.p.per_group * a.p.part_rows;
        int64_t r1 = (group + 1) * a.p.group_rows;
        r1 = r1 < r0 + a.p.part_rows ? r1 : r0 + a.p.part_rows;
        r1 = r1 < a.T ? r1 : a.T;
        const uint4* gr = gate_row(a.gate, a.gate_rows, r0, a.vecs);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            gv[i] = gr && c < a.vecs ? gr[c] : none;
        }
        for (int64_t row = r0; row < r1; ++row, turn ^= 1) {
            const int64_t base = row * a.vecs;
            const float tg = token_gate<BF16>(a.gate, a.gate_rows, row);
            const float rs1 = a.w_post ? a.rstd_post[row] : 1.0f, rs2 = a.dy ? a.rstd_pre[row] : 0.0f;
            uint4 ux[CH], us[CH], ud[CH], ue[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = i * blockDim.x + threadIdx.x;
                ux[i] = us[i] = ud[i] = ue[i] = none;
                if (c < a.vecs) {
                    ux[i] = moe::load16<STREAM>(a.x + base + c);
                    if (a.dy) {
                        us[i] = moe::load16<STREAM>(a.s + base + c);
                        ud[i] = moe::load16<STREAM>(a.dy + base + c);
                    }
                    if (a.ds) ue[i] = moe::load16<STREAM>(a.ds + base + c);
                }
            }
            float d[CH][N], dot = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) V::load(ue[i], d[i]);
            if (a.dy) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    float sv[N], g[N], w[N];
                    V::load(us[i], sv);
                    V::load(ud[i], g);
                    V::load(w2[i], w);
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const float sh = sv[k] * rs2;
                        acc_pre[i][k] = fmaf(g[k], sh, acc_pre[i][k]);
                        dot = fmaf(g[k] * w[k], sh, dot);
                    }
                }
                const float mean = wg_sum(dot, red[turn][0]) * inv_h;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    float sv[N], g[N], w[N];
                    V::load(us[i], sv);
                    V::load(ud[i], g);
                    V::load(w2[i], w);
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        d[i][k] = fmaf(rs2, fmaf(-(sv[k] * rs2), mean, g[k] * w[k]), d[i][k]);
                }
            }
            if (a.dresidual)
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int c = i * blockDim.x + threadIdx.x;
                    float v[N];
#pragma unroll
                    for (int k = 0; k < N; ++k) v[k] = a.alpha * d[i][k];
                    if (c < a.vecs) moe::store16<STREAM>(a.dresidual + base + c, V::store(v));
                }
            // xhat (x without a norm behind) and what reaches it
            dot = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float x[N], w[N], g[N];
                V::load(ux[i], x);
                V::load(w1[i], w);
                V::load(gv[i], g);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float xh = x[k] * rs1, n = a.w_post ? xh * w[k] : xh;
                    acc_gate[i][k] = fmaf(d[i][k], n, acc_gate[i][k]);
                    const float dn = gr ? d[i][k] * g[k] : d[i][k];  // (a token's gate follows)
                    acc_post[i][k] = fmaf(dn * tg, xh, acc_post[i][k]);
                    dot = fmaf(gr ? dn * w[k] : d[i][k], gr ? xh : n, dot);
                    d[i][k] = dn * tg;
                }
            }
            float mean = 0.0f;
            if (a.w_post || a.token_dgate) {
                // without a row of gates: sum d n, a token's dgate; it times the gate is
                // the sum that dx needs
                dot = wg_sum(dot, red[turn][1]);
                if (a.token_dgate && threadIdx.x == 0) a.token_dgate[row] = dot;
                mean = a.w_post ? dot * tg * inv_h : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = i * blockDim.x + threadIdx.x;
                float x[N], w[N];
                V::load(ux[i], x);
                V::load(w1[i], w);
                if (a.w_post)
#pragma unroll
                    for (int k = 0; k < N; ++k) d[i][k] = rs1 * fmaf(-(x[k] * rs1), mean, d[i][k] * w[k]);
                if (c < a.vecs) moe::store16<STREAM>(a.dx + base + c, V::store(d[i]));
            }
        }
        if (a.part_gate)
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = i * blockDim.x + threadIdx.x;
                if (c < a.vecs) store_sums<N>(a.part_gate + part * a.H + (int64_t)c * N, acc_gate[i]);
#pragma unroll
                for (int k = 0; k < N; ++k) acc_gate[i][k] = 0.0f;
            }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        const int64_t at = (int64_t)blockIdx.x * a.H + (int64_t)c * N;
        if (c < a.vecs && a.part_post) store_sums<N>(a.part_post + at, acc_post[i]);
        if (c < a.vecs && a.part_pre) store_sums<N>(a.part_pre + at, acc_pre[i]);
    }
}

// Rows too wide for the registers: the sums are kept in the workspace, d is
// computed again where it is needed.
template <bool BF16>
__global__ __launch_bounds__(kMaxThreads) void block_norm_bwd_wide_kernel(const Bwd a)
{
    using V = Vec<BF16>;
    constexpr int N = V::kN;
    __shared__ float red[2][2][16];
    const float inv_h = 1.0f / (float)a.H;
    const uint4 none = make_uint4(0, 0, 0, 0);
    const int64_t mine = (int64_t)blockIdx.x * a.H;
    // (each thread adds to its own columns; a group's last parts may have no rows)
    auto clear = [&](float* sums) {
        for (int c = threadIdx.x; sums && c < a.vecs; c += blockDim.x)
#pragma unroll
            for (int k = 0; k < N; ++k) sums[(int64_t)c * N + k] = 0.0f;
    };
    clear(a.part_post ? a.part_post + mine : nullptr);
    clear(a.part_pre ? a.part_pre + mine : nullptr);
    int turn = 0;
    for (int64_t part = blockIdx.x; part < a.p.parts; part += gridDim.x) {
        const int64_t group = part / a.p.per_group, r0 = group * a.p.group_rows + part % a.p.per_group * a.p.part_rows;
        int64_t r1 = (group + 1) * a.p.group_rows;
        r1 = r1 < r0 + a.p.part_rows ? r1 : r0 + a.p.part_rows;
        r1 = r1 < a.T ? r1 : a.T;
        const uint4* gr = gate_row(a.gate, a.gate_rows, r0, a.vecs);
        clear(a.part_gate ? a.part_gate + part * a.H : nullptr);
        for (int64_t row = r0; row < r1; ++row, turn ^= 1) {
            const int64_t base = row * a.vecs;
            const float tg = token_gate<BF16>(a.gate, a.gate_rows, row);
            const float rs1 = a.w_post ? a.rstd_post[row] : 1.0f, rs2 = a.dy ? a.rstd_pre[row] : 0.0f;
            float dot = 0.0f, mean1 = 0.0f;
            if (a.dy) {
                for (int c = threadIdx.x; c < a.vecs; c += blockDim.x) {
                    float sv[N], g[N], w[N];
                    V::load(a.s[base + c], sv);
                    V::load(a.dy[base + c], g);
                    V::load(a.w_pre[c], w);
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const float sh = sv[k] * rs2;
                        if (a.part_pre) {
                            float* p = a.part_pre + mine + (int64_t)c * N + k;
                            *p = fmaf(g[k], sh, *p);
                        }
                        dot = fmaf(g[k] * w[k], sh, dot);
                    }
                }
                mean1 = wg_sum(dot, red[turn][0]) * inv_h;
            }
            auto d_at = [&](int c, float* d) {
                V::load(a.ds ? a.ds[base + c] : none, d);
                if (!a.dy) return;
                float sv[N], g[N], w[N];
                V::load(a.s[base + c], sv);
                V::load(a.dy[base + c], g);
                V::load(a.w_pre[c], w);
#pragma unroll
                for (int k = 0; k < N; ++k) d[k] = fmaf(rs2, fmaf(-(sv[k] * rs2), mean1, g[k] * w[k]), d[k]);
            };
            dot = 0.0f;
            for (int c = threadIdx.x; c < a.vecs; c += blockDim.x) {
                float d[N], x[N], w[N], g[N];
                d_at(c, d);
                V::load(a.x[base + c], x);
                V::load(a.w_post ? a.w_post[c] : none, w);
                V::load(gr ? gr[c] : none, g);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float xh = x[k] * rs1, n = a.w_post ? xh * w[k] : xh;
                    const float dn = gr ? d[k] * g[k] : d[k];
                    if (a.part_gate) {
                        float* p = a.part_gate + part * a.H + (int64_t)c * N + k;
                        *p = fmaf(d[k], n, *p);
                    }
                    if (a.part_post) {
                        float* p = a.part_post + mine + (int64_t)c * N + k;
                        *p = fmaf(dn * tg, xh, *p);
                    }
                    dot = fmaf(gr ? dn * w[k] : d[k], gr ? xh : n, dot);
                }
            }
            float mean2 = 0.0f;
            if (a.w_post || a.token_dgate) {
                dot = wg_sum(dot, red[turn][1]);
                if (a.token_dgate && threadIdx.x == 0) a.token_dgate[row] = dot;
                mean2 = a.w_post ? dot * tg * inv_h : 0.0f;
            }
            // (dx or dresidual may be dy or ds: a vector is stored after its last reading)
            for (int c = threadIdx.x; c < a.vecs; c += blockDim.x) {
                float d[N], x[N], w[N], g[N], v[N];
                d_at(c, d);
                V::load(a.x[base + c], x);
                V::load(a.w_post ? a.w_post[c] : none, w);
                V::load(gr ? gr[c] : none, g);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float dn = (gr ? d[k] * g[k] : d[k]) * tg;
                    v[k] = a.w_post ? rs1 * fmaf(-(x[k] * rs1), mean2, dn * w[k]) : dn;
                    d[k] *= a.alpha;
                }
                if (a.dresidual) a.dresidual[base + c] = V::store(d);
                a.dx[base + c] = V::store(v);
            }
        }
    }
}

// Sums over the parts in a fixed order: 16 threads per column take every 16th
// part, then their sums are added in order. blockIdx.y: dw_post, dw_pre, then the
// groups of the gate.
struct Sums {
    int H, G, per_group;
    const float *part_post, *part_pre, *part_gate;
    float *dw_post, *dw_pre, *dgate;
};
__global__ __launch_bounds__(1024) void block_norm_sums_kernel(const Sums a, int h0)
{
    __shared__ float sh[16][kRedCols];
    const int which = blockIdx.y;
    const int64_t group = which - 2;
    const float* from = which == 0 ? a.part_post : which == 1 ? a.part_pre
                                   : a.part_gate + group * a.per_group * a.H;
    float* to = which == 0 ? a.dw_post : which == 1 ? a.dw_pre : a.dgate + group * a.H;
    const int n = which < 2 ? a.G : a.per_group;
    if (which < 2 && !to) return;
    const int col = threadIdx.x % kRedCols, grp = threadIdx.x / kRedCols;
    const int h = h0 + blockIdx.x * kRedCols + col;
    float v = 0.0f;
    if (h < a.H) {
        int g = grp;
        for (; g + 7 * 16 < n; g += 8 * 16) {  // eight loads in flight
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = from[(int64_t)(g + 16 * i) * a.H + h];
#pragma unroll
            for (int i = 0; i < 8; ++i) v += t[i];
        }
        for (; g < n; g += 16) v += from[(int64_t)g * a.H + h];
    }
    sh[grp][col] = v;
    __syncthreads();
    if (grp == 0 && h < a.H) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += sh[i][col];
        to[h] = t;
    }
}

__global__ __launch_bounds__(256) void block_norm_zero_kernel(float* a, float* b, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        if (a) a[i] = 0.0f;
        if (b) b[i] = 0.0f;
    }
}

// ----------------------------------------------------------------- launches --

// As moe_rmsnorm: at most four vectors a thread on up to 1024 threads (of x and
// of the residual), else the wide kernel.
template <bool BF16, bool STREAM>
hipError_t launch_fwd(const Fwd& a, int rows, hipStream_t st)
{
    int t = a.vecs <= 64 ? 64 : a.vecs <= 128 ? 128 : 256;
    while (t < kMaxThreads && a.vecs > 4 * t) t *= 2;
    switch ((a.vecs + t - 1) / t) {
#define MOE_NORM(C)                                                     \
    case C:                                                             \
        block_norm_kernel<BF16, C, STREAM><<<rows, t, 0, st>>>(a);      \
        break;
        MOE_NORM(1) MOE_NORM(2) MOE_NORM(3) MOE_NORM(4)
#undef MOE_NORM
    default:
        block_norm_wide_kernel<BF16><<<rows, kMaxThreads, 0, st>>>(a);
    }
    return hipGetLastError();
}

template <bool BF16, bool STREAM>
hipError_t launch_bwd(const Bwd& a, hipStream_t st)
{
    int t = 64;
    while (t < 512 && a.vecs > 2 * t) t *= 2;
    const int ch = (a.vecs + t - 1) / t, G = a.p.grid;
    if (ch == 1) block_norm_bwd_kernel<BF16, 1, 512, STREAM><<<G, t, 0, st>>>(a);
    else if (ch == 2) block_norm_bwd_kernel<BF16, 2, 512, STREAM><<<G, t, 0, st>>>(a);
    else block_norm_bwd_wide_kernel<BF16><<<G, kMaxThreads, 0, st>>>(a);
    return hipGetLastError();
}

template <typename T>
const uint4* vec(const T* p)
{
    return reinterpret_cast<const uint4*>(p);
}

}  // namespace

hipError_t moe_launch_block_norm(const moe_shape_t& s, const MoeBlockNorm& m, hipStream_t st)
{
    const bool bf = s.dtype == MOE_BF16;
    const int64_t row = (int64_t)s.H * (bf ? 2 : 4);
    const bool stream = s.T * (row * (1 + !!m.residual + !!m.s + !!m.y) + (m.q ? s.H : 0)) > moe::kStreamBytes;
    Fwd a{s.H, s.H / (bf ? 8 : 4), 0, vec(m.x), vec(m.residual), m.alpha, m.eps, vec(m.w_post), vec(m.w_pre),
          m.gate, (uint32_t)m.gate_rows, static_cast<uint4*>(m.s), static_cast<uint4*>(m.y), static_cast<uint8_t*>(m.q),
          static_cast<uint8_t*>(m.scales), m.rstd_post, m.rstd_pre};
    auto* launch = bf ? (stream ? launch_fwd<true, true> : launch_fwd<true, false>)
                      : (stream ? launch_fwd<false, true> : launch_fwd<false, false>);
    for (int64_t t0 = 0; t0 < s.T; t0 += kMaxRows) {
        a.row0 = t0;
        const hipError_t e = launch(a, (int)(s.T - t0 < kMaxRows ? s.T - t0 : kMaxRows), st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t moe_launch_block_norm_backward(const moe_shape_t& s, const MoeBlockNormBwd& m, float* ws, hipStream_t st)
{
    const bool bf = s.dtype == MOE_BF16, rows_gate = m.gate && m.gate_rows > 0 && m.dgate;
    const int32_t gate_rows = m.gate ? m.gate_rows : 0;
    const moe::BlockNormParts p = moe::block_norm_parts(s.T, gate_rows);
    if (s.T == 0) {  // sums over no rows
        if (!m.dw_post && !m.dw_pre) return hipSuccess;
        block_norm_zero_kernel<<<(s.H + 255) / 256 < 1024 ? (s.H + 255) / 256 : 1024, 256, 0, st>>>(m.dw_post, m.dw_pre, s.H);
        return hipGetLastError();
    }
    Bwd a{s.H, s.H / (bf ? 8 : 4), s.T, p, vec(m.x), vec(m.s), vec(m.w_post), vec(m.w_pre), vec(m.dy), vec(m.ds),
          m.rstd_post, m.rstd_pre, m.alpha, m.gate, (uint32_t)gate_rows, static_cast<uint4*>(m.dx), static_cast<uint4*>(m.dresidual),
          m.gate && !gate_rows ? m.dgate : nullptr, nullptr, nullptr, nullptr};
    if (m.dw_post) a.part_post = ws;
    if (m.dw_pre) a.part_pre = ws + (int64_t)p.grid * s.H;
    if (rows_gate) a.part_gate = p.per_group > 1 ? ws + 2 * (int64_t)p.grid * s.H : m.dgate;
    const int64_t row = (int64_t)s.H * (bf ? 2 : 4);
    const bool stream = s.T * row * (2 + !!m.ds + !!m.dresidual + 2 * !!m.dy) > moe::kStreamBytes;
    auto* launch = bf ? (stream ? launch_bwd<true, true> : launch_bwd<true, false>)
                      : (stream ? launch_bwd<false, true> : launch_bwd<false, false>);
    hipError_t e = launch(a, st);
    if (e != hipSuccess) return e;
    // (groups of several parts are fewer than kNormBwdGroups)
    const int groups = rows_gate && p.per_group > 1 ? (int)p.groups : 0;
    if (!m.dw_post && !m.dw_pre && !groups) return hipSuccess;
    const Sums q{s.H, p.grid, p.per_group, a.part_post, a.part_pre, a.part_gate, m.dw_post, m.dw_pre, m.dgate};
    for (int64_t h0 = 0; h0 < s.H; h0 += (int64_t)2048 * kRedCols) {
        const int64_t left = (s.H - h0 + kRedCols - 1) / kRedCols;
        block_norm_sums_kernel<<<dim3((unsigned)(left < 2048 ? left : 2048), 2 + groups), 1024, 0, st>>>(q, (int)h0);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}
