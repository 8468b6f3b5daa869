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
// CH 16-byte vectors of x and of the residual per thread. The sums of squares are
// fp64 (hidden under the memory traffic), all else fp32; s is rounded to the type
// before its norm, so that y is the norm of what the next block reads as its stream.
//
// Measured: forward of 8192 x 7168 in bf16 with s, y and 8-bit blocks (530 MB) 91 us in
// a stream of calls on buffers that stay, 5.8 TB/s, 95 to 101 where inputs and outputs
// alternate; in fp32 (940 MB) 159 us, 5.9 TB/s; of one row of 4096 4.3 us. Backward of
// 8192 x 7168 in bf16 with both gradients and a gate (705 MB) 130 to 132 us, 5.4 TB/s, and
// 5 us for the sums.
#include "lanes.h"
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
//   d = ds + rstd_pre (g - shat m), g = dy w_pre, shat = s rstd_pre, m = mean(g shat);
//   dresidual = alpha d, dn = gate d,
//   dx = rstd_post (e - xhat mean(e xhat)), e = dn w_post, xhat = x rstd_post.
// The second mean needs d, and with it the first one; taken apart it does not:
//   sum(e xhat) = sum(a (ds + rstd_pre g)) - m sum(a rstd_pre shat), a = gate w_post xhat,
// so that a row's three sums meet at one barrier.
//
// A workgroup takes parts (every n-th row under one row of gates) b, b + G, ...
// and keeps the fp32 sums of dw_pre and dw_post of its columns over all of its
// rows, and those of dgate over a part, so that the sums' order is fixed. The next
// row is loaded while one is summed.
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

// Three sums over the workgroup, in a fixed order. red: LDS that the row before
// does not use.
__device__ __forceinline__ void sum3(float (&v)[3], float (*red)[16])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = moe::lanes::group_reduce<64, true>(v[i]);
    const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < 3; ++i) red[i][wave] = v[i];
    __syncthreads();
    const int w = threadIdx.x & 15;  // (every 16 lanes add the waves' up: one read, four steps)
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = red[i][w];
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = moe::lanes::group_reduce<16, true>(w < waves ? v[i] : 0.0f);
}

// A part's rows: r0, r0 + per_group, ... below r1.
struct Rows {
    int64_t r0, r1;
};
__device__ __forceinline__ Rows rows_of(const Bwd& a, int64_t part)
{
    const int64_t group = part / a.p.per_group, r1 = (group + 1) * a.p.group_rows;
    return Rows{group * a.p.group_rows + part % a.p.per_group, r1 < a.T ? r1 : a.T};
}

// dw_post and dgate are one sum over a part's rows, A = sum(token's gate * d xhat),
// times a column's gate and times its weight.
template <bool BF16, int CH, int TH, bool STREAM>
__global__ __launch_bounds__(TH) void block_norm_bwd_kernel(const Bwd a)
{
    using V = Vec<BF16>;
    constexpr int N = V::kN;
    __shared__ float red[2][3][16];
    const float inv_h = 1.0f / (float)a.H;
    const uint4 none = make_uint4(0, 0, 0, 0);
    float acc[CH][N], acc_post[CH][N], acc_pre[CH][N];
    float w2[CH][N], gw[CH][N];  // w_pre, gate * w_post
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        V::load(c < a.vecs && a.w_pre ? a.w_pre[c] : none, w2[i]);
#pragma unroll
        for (int k = 0; k < N; ++k) acc[i][k] = acc_post[i][k] = acc_pre[i][k] = 0.0f;
    }
    uint4 nx[CH], ns[CH], nd[CH], ne[CH];  // the next row
    float n1 = 1.0f, n2 = 0.0f, ng = 1.0f;
    auto load = [&](int64_t row) {
        if (a.w_post) n1 = a.rstd_post[row];
        if (a.dy) n2 = a.rstd_pre[row];
        ng = token_gate<BF16>(a.gate, a.gate_rows, row);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            const int64_t at = row * a.vecs + c;
            nx[i] = ns[i] = nd[i] = ne[i] = none;
            if (c < a.vecs) {
                nx[i] = moe::load16<STREAM>(a.x + at);
                if (a.dy) {
                    ns[i] = moe::load16<STREAM>(a.s + at);
                    nd[i] = moe::load16<STREAM>(a.dy + at);
                }
                if (a.ds) ne[i] = moe::load16<STREAM>(a.ds + at);
            }
        }
    };
    // this thread's columns of w_post and of the part's gates (1 where there is none)
    auto column = [&](const uint4* from, int i, float* v) {
        const int c = i * blockDim.x + threadIdx.x;
        if (from) V::load(c < a.vecs ? from[c] : none, v);
        else
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = 1.0f;
    };
    int turn = 0;
    for (int64_t part = blockIdx.x; part < a.p.parts; part += gridDim.x) {
        const Rows rows = rows_of(a, part);
        const uint4* gr = gate_row(a.gate, a.gate_rows, rows.r0, a.vecs);
        if (rows.r0 < rows.r1) load(rows.r0);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float w[N], g[N];
            column(a.w_post, i, w);
            column(gr, i, g);
#pragma unroll
            for (int k = 0; k < N; ++k) gw[i][k] = g[k] * w[k];
        }
        for (int64_t row = rows.r0; row < rows.r1; row += a.p.per_group, turn ^= 1) {
            const int64_t base = row * a.vecs;
            const float tg = ng, rs1 = n1, rs2 = n2;
            // xhat, shat, and d but for the first mean
            float xh[CH][N], sh[CH][N], d[CH][N], sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float dy[N];
                V::load(nx[i], xh[i]);
                V::load(ns[i], sh[i]);
                V::load(nd[i], dy);
                V::load(ne[i], d[i]);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    xh[i][k] *= rs1;
                    sh[i][k] *= rs2;
                    const float g = dy[k] * w2[i][k], p = xh[i][k] * gw[i][k];
                    acc_pre[i][k] = fmaf(dy[k], sh[i][k], acc_pre[i][k]);
                    d[i][k] = fmaf(rs2, g, d[i][k]);
                    sum[0] = fmaf(g, sh[i][k], sum[0]);
                    sum[1] = fmaf(p, d[i][k], sum[1]);
                    sum[2] = fmaf(p, sh[i][k], sum[2]);
                }
            }
            // (dx or dresidual may be dy or ds: this row is in registers before it is
            // stored, and the next one is another)
            if (row + a.p.per_group < rows.r1) load(row + a.p.per_group);
            sum3(sum, red[turn]);
            const float m = sum[0] * inv_h * rs2, dot = fmaf(-m, sum[2], sum[1]);
            // without a row of gates dot is sum(d n): a token's dgate
            if (a.token_dgate && threadIdx.x == 0) a.token_dgate[row] = dot;
            const float r = tg * rs1, mean = a.w_post ? dot * inv_h : 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = i * blockDim.x + threadIdx.x;
                float v[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float dk = fmaf(-m, sh[i][k], d[i][k]);
                    acc[i][k] = fmaf(tg * dk, xh[i][k], acc[i][k]);
                    v[k] = r * fmaf(-mean, xh[i][k], dk * gw[i][k]);
                    d[i][k] = a.alpha * dk;
                }
                if (c < a.vecs) {
                    if (a.dresidual) moe::store16<STREAM>(a.dresidual + base + c, V::store(d[i]));
                    moe::store16<STREAM>(a.dx + base + c, V::store(v));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            float w[N], g[N];
            column(a.w_post, i, w);
            column(gr, i, g);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                acc_post[i][k] = fmaf(g[k], acc[i][k], acc_post[i][k]);
                w[k] *= acc[i][k];
                acc[i][k] = 0.0f;
            }
            if (a.part_gate && c < a.vecs) store_sums<N>(a.part_gate + part * a.H + (int64_t)c * N, w);
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

// Rows too wide for the registers: the sums are kept in the workspace, two passes
// over the row.
template <bool BF16>
__global__ __launch_bounds__(kMaxThreads) void block_norm_bwd_wide_kernel(const Bwd a)
{
    using V = Vec<BF16>;
    constexpr int N = V::kN;
    __shared__ float red[2][3][16];
    const float inv_h = 1.0f / (float)a.H;
    const uint4 none = make_uint4(0, 0, 0, 0);
    const int64_t mine = (int64_t)blockIdx.x * a.H;
    // (each thread adds to its own columns; a group's last parts may have no rows)
    auto clear = [&](float* sums) {
        for (int c = threadIdx.x; sums && c < a.vecs; c += blockDim.x)
#pragma unroll
            for (int k = 0; k < N; ++k) sums[(int64_t)c * N + k] = 0.0f;
    };
    auto add = [&](float* sums, int c, const float* v) {
        if (!sums) return;
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            float4* p = reinterpret_cast<float4*>(sums + (int64_t)c * N + k);
            const float4 o = *p;
            *p = make_float4(o.x + v[k], o.y + v[k + 1], o.z + v[k + 2], o.w + v[k + 3]);
        }
    };
    clear(a.part_post ? a.part_post + mine : nullptr);
    clear(a.part_pre ? a.part_pre + mine : nullptr);
    int turn = 0;
    for (int64_t part = blockIdx.x; part < a.p.parts; part += gridDim.x) {
        const Rows rows = rows_of(a, part);
        const uint4* gr = gate_row(a.gate, a.gate_rows, rows.r0, a.vecs);
        clear(a.part_gate ? a.part_gate + part * a.H : nullptr);
        for (int64_t row = rows.r0; row < rows.r1; row += a.p.per_group, turn ^= 1) {
            const int64_t base = row * a.vecs;
            const float tg = token_gate<BF16>(a.gate, a.gate_rows, row);
            const float rs1 = a.w_post ? a.rstd_post[row] : 1.0f, rs2 = a.dy ? a.rstd_pre[row] : 0.0f;
            float x[N], sv[N], dy[N], d[N], w[N], v[N], g[N], sum[3] = {0.0f, 0.0f, 0.0f};
            auto load = [&](int c) {
                V::load(a.x[base + c], x);
                V::load(a.dy ? a.s[base + c] : none, sv);
                V::load(a.dy ? a.dy[base + c] : none, dy);
                V::load(a.ds ? a.ds[base + c] : none, d);
                V::load(a.w_post ? a.w_post[c] : none, w);
                V::load(a.w_pre ? a.w_pre[c] : none, v);
                V::load(gr ? gr[c] : none, g);
            };
            for (int c = threadIdx.x; c < a.vecs; c += blockDim.x) {
                load(c);
                float pre[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float xh = x[k] * rs1, sh = sv[k] * rs2, gd = dy[k] * v[k];
                    const float n = a.w_post ? xh * w[k] : xh, p = gr ? n * g[k] : n;
                    pre[k] = dy[k] * sh;
                    sum[0] = fmaf(gd, sh, sum[0]);
                    sum[1] = fmaf(p, fmaf(rs2, gd, d[k]), sum[1]);
                    sum[2] = fmaf(p, rs2 * sh, sum[2]);
                }
                add(a.part_pre ? a.part_pre + mine : nullptr, c, pre);
            }
            sum3(sum, red[turn]);
            const float m = sum[0] * inv_h, dot = fmaf(-m, sum[2], sum[1]), mean = dot * tg * inv_h;
            if (a.token_dgate && threadIdx.x == 0) a.token_dgate[row] = dot;
            // (dx or dresidual may be dy or ds: a vector is stored after its last reading)
            for (int c = threadIdx.x; c < a.vecs; c += blockDim.x) {
                load(c);
                float gate[N], post[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float xh = x[k] * rs1;
                    d[k] = fmaf(rs2, fmaf(-(sv[k] * rs2), m, dy[k] * v[k]), d[k]);
                    gate[k] = d[k] * (a.w_post ? xh * w[k] : xh);
                    const float dn = d[k] * (gr ? g[k] : tg);
                    post[k] = dn * xh;
                    v[k] = a.w_post ? rs1 * fmaf(-xh, mean, dn * w[k]) : dn;
                    d[k] *= a.alpha;
                }
                add(a.part_gate ? a.part_gate + part * a.H : nullptr, c, gate);
                add(a.part_post ? a.part_post + mine : nullptr, c, post);
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

// One vector a thread; two of fp32, whose kernel spills 28 vector registers; two of bf16
// spill 182, and the wide kernel takes those rows. One gate a channel, us, two vectors
// and wide: bf16 8192 x 8256 844 and 626, 8192 x 16384 1215 and 1177, 1024 x 12288 168 and
// 124; fp32 8192 x 4160 172 and 487, 8192 x 8192 301 and 928, 1024 x 7168 60 and 111.
template <bool BF16, bool STREAM>
hipError_t launch_bwd(const Bwd& a, hipStream_t st)
{
    const int G = a.p.grid, t = (a.vecs + 63) / 64 * 64;
    if (t <= 512) {
        block_norm_bwd_kernel<BF16, 1, 512, STREAM><<<G, t, 0, st>>>(a);
        return hipGetLastError();
    }
    if (t <= 1024) {
        block_norm_bwd_kernel<BF16, 1, 1024, STREAM><<<G, t, 0, st>>>(a);
        return hipGetLastError();
    }
    if constexpr (!BF16)
        if (t <= 2048) {
            block_norm_bwd_kernel<BF16, 2, 1024, STREAM><<<G, (a.vecs + 127) / 128 * 64, 0, st>>>(a);
            return hipGetLastError();
        }
    block_norm_bwd_wide_kernel<BF16><<<G, kMaxThreads, 0, st>>>(a);
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
    const moe::BlockNormParts p = moe::block_norm_parts(s, gate_rows);
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
    // (groups of several parts are fewer than the workgroups, 1024 at most)
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
