// norm.hip -- the root-mean-square norm in front of the layer, with the
// residual's addition and an output in 8-bit blocks, and its backward.
//
//   s = round(x + residual), rstd = (mean s^2 + eps)^-1/2, v = s rstd weight,
//   y = round(v), (q, scales) = blocks(v).
//
// Bound by memory: each input is read once and each output written once. One
// workgroup takes one row and keeps it in registers between the sum of
// squares and the outputs, as CH 16-byte vectors per thread: at most 256
// threads where four vectors a thread hold the row, so that several rows share
// a CU and one row's loads cover another's sum.
//
// Measured: forward, 8192 rows of 7168 bf16 with residual, y and 8-bit output,
// 86 us (6.2 TB/s; a plain copy of 2 GiB reaches 4.9, a read 6.2), 96 us through
// the caches; backward of the same, 82 us (91) + 5 us for dweight's sum (5.4
// TB/s); one row of 4096, 3 us.
#include <type_traits>

#include "rows.h"

namespace {

using moe::rows::Vec;
using moe::rows::rstd_of;
using moe::rows::store_mx;
using moe::rows::wg_sum;

constexpr int kMaxCh = 4;          // vectors per thread on the register path
constexpr int kMaxThreads = 1024;
constexpr int kMaxRows = 1 << 21;  // workgroups of a launch: of kMaxThreads each, half of the 2^32 threads it can hold
constexpr int kRedCols = 64;       // columns per workgroup of the dweight sum

// s = round(x + residual) of one vector (the stored value is the normed one)
template <bool BF16>
__device__ __forceinline__ void add_residual(uint4& u, const uint4& r, float* f)
{
    using V = Vec<BF16>;
    float b[V::kN];
    V::load(u, f);
    V::load(r, b);
#pragma unroll
    for (int k = 0; k < V::kN; ++k) f[k] += b[k];
    u = V::store(f);
    V::load(u, f);
}

// s, y may be x or residual: a thread stores a vector only after it read it
template <bool BF16, int CH, bool STREAM>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_kernel(int H, int vecs, const uint4* x,
                                                              const uint4* residual,
                                                              const uint4* __restrict__ weight, float eps,
                                                              uint4* s, uint4* y, uint8_t* q,
                                                              uint8_t* scales, float* rstd)
{
    using V = Vec<BF16>;
    __shared__ double red[16];
    const int64_t row = blockIdx.x, base = row * vecs;
    uint4 u[CH], r[CH], wv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        u[i] = make_uint4(0, 0, 0, 0);
        wv[i] = u[i];
        if (c < vecs) {
            u[i] = moe::load16<STREAM>(x + base + c);
            if (residual) r[i] = moe::load16<STREAM>(residual + base + c);
            wv[i] = weight[c];
        }
    }
    float f[CH][V::kN];
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (residual && c < vecs) add_residual<BF16>(u[i], r[i], f[i]);
        else V::load(u[i], f[i]);
        if (s && c < vecs) moe::store16<STREAM>(s + base + c, u[i]);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) ss = fma((double)f[i][k], (double)f[i][k], ss);
    }
    const float rs = rstd_of(wg_sum(ss, red), H, eps);
    if (rstd && threadIdx.x == 0) rstd[row] = rs;
    if (!y && !q) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        float w[V::kN];
        V::load(wv[i], w);
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[i][k] = f[i][k] * rs * w[k];
        if (y && c < vecs) moe::store16<STREAM>(y + base + c, V::store(f[i]));
        if (q) store_mx<BF16>(f[i], base + c, c < vecs, q, scales);
    }
}

// Rows too wide for the registers: two passes over the row.
template <bool BF16>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_wide_kernel(int H, int vecs, const uint4* x,
                                                                   const uint4* residual,
                                                                   const uint4* __restrict__ weight,
                                                                   float eps, uint4* s, uint4* y,
                                                                   uint8_t* q, uint8_t* scales, float* rstd)
{
    using V = Vec<BF16>;
    __shared__ double red[16];
    const int64_t row = blockIdx.x, base = row * vecs;
    double ss = 0.0;
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
        float f[V::kN];
        uint4 u = x[base + c];
        if (residual) add_residual<BF16>(u, residual[base + c], f);
        else V::load(u, f);
        if (s) s[base + c] = u;
#pragma unroll
        for (int k = 0; k < V::kN; ++k) ss = fma((double)f[k], (double)f[k], ss);
    }
    const float rs = rstd_of(wg_sum(ss, red), H, eps);
    if (rstd && threadIdx.x == 0) rstd[row] = rs;
    if (!y && !q) return;
    // s, where it is kept, may have replaced x or residual: read it back then
    for (int c0 = 0; c0 < vecs; c0 += blockDim.x) {
        const int c = c0 + threadIdx.x;
        float f[V::kN], w[V::kN];
#pragma unroll
        for (int k = 0; k < V::kN; ++k) f[k] = 0.0f;
        if (c < vecs) {
            uint4 u = s ? s[base + c] : x[base + c];
            if (residual && !s) add_residual<BF16>(u, residual[base + c], f);
            else V::load(u, f);
            V::load(weight[c], w);
#pragma unroll
            for (int k = 0; k < V::kN; ++k) f[k] = f[k] * rs * w[k];
            if (y) y[base + c] = V::store(f);
        }
        if (q) store_mx<BF16>(f, base + c, c < vecs, q, scales);
    }
}

// One row of the backward in registers: dx, and this row's part of dweight
// added to acc.
//   xhat = s rstd, g = dy weight, dx = rstd (g - xhat mean(g xhat)) + ds.
// Workgroup b takes rows b, b + G, ...; each thread keeps the fp32 sums of
// its columns over those rows and writes them to part[b], so that the sum's
// order is fixed.
template <bool BF16, int CH, int TH, bool STREAM>
__global__ __launch_bounds__(TH) void rmsnorm_bwd_kernel(int T, int H, int vecs, const uint4* s,
                                                                  const uint4* __restrict__ weight,
                                                                  const float* __restrict__ rstd,
                                                                  const uint4* dy, const uint4* ds,
                                                                  uint4* dx, float* __restrict__ part)
{
    using V = Vec<BF16>;
    __shared__ float red[2][16];
    const float inv_h = 1.0f / (float)H;
    float acc[CH][V::kN];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int k = 0; k < V::kN; ++k) acc[i][k] = 0.0f;
    uint4 wv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        wv[i] = c < vecs ? weight[c] : make_uint4(0, 0, 0, 0);
    }
    int turn = 0;
    for (int row = blockIdx.x; row < T; row += gridDim.x, turn ^= 1) {
        const int64_t base = (int64_t)row * vecs;
        const float rs = rstd[row];
        uint4 us[CH], ud[CH], ue[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            us[i] = make_uint4(0, 0, 0, 0);
            ud[i] = us[i];
            ue[i] = us[i];
            if (c < vecs) {
                us[i] = moe::load16<STREAM>(s + base + c);
                ud[i] = moe::load16<STREAM>(dy + base + c);
                if (ds) ue[i] = moe::load16<STREAM>(ds + base + c);
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float a[V::kN], d[V::kN], w[V::kN];
            V::load(us[i], a);
            V::load(ud[i], d);
            V::load(wv[i], w);
#pragma unroll
            for (int k = 0; k < V::kN; ++k) {
                const float xh = a[k] * rs;
                acc[i][k] = fmaf(d[k], xh, acc[i][k]);
                dot = fmaf(d[k] * w[k], xh, dot);
            }
        }
        const float mean = wg_sum(dot, red[turn]) * inv_h;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            float a[V::kN], d[V::kN], w[V::kN], e[V::kN];
            V::load(us[i], a);
            V::load(ud[i], d);
            V::load(wv[i], w);
            V::load(ue[i], e);
#pragma unroll
            for (int k = 0; k < V::kN; ++k)
                e[k] = fmaf(rs, fmaf(-(a[k] * rs), mean, d[k] * w[k]), e[k]);
            if (c < vecs) moe::store16<STREAM>(dx + base + c, V::store(e));
        }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c < vecs)
#pragma unroll
            for (int k = 0; k < V::kN; k += 4)
                *reinterpret_cast<float4*>(part + (int64_t)blockIdx.x * H + (int64_t)c * V::kN + k) =
                    make_float4(acc[i][k], acc[i][k + 1], acc[i][k + 2], acc[i][k + 3]);
    }
}

template <bool BF16>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_bwd_wide_kernel(
    int T, int H, int vecs, const uint4* s, const uint4* __restrict__ weight,
    const float* __restrict__ rstd, const uint4* dy, const uint4* ds, uint4* dx, float* part)
{
    using V = Vec<BF16>;
    __shared__ float red[2][16];
    float* mine = part + (int64_t)blockIdx.x * H;
    int turn = 0;
    for (int row = blockIdx.x; row < T; row += gridDim.x, turn ^= 1) {
        const int64_t base = (int64_t)row * vecs;
        const float rs = rstd[row];
        const bool first = row == (int)blockIdx.x;
        float dot = 0.0f;
        for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
            float a[V::kN], d[V::kN], w[V::kN];
            V::load(s[base + c], a);
            V::load(dy[base + c], d);
            V::load(weight[c], w);
#pragma unroll
            for (int k = 0; k < V::kN; ++k) {
                const float xh = a[k] * rs;
                float* p = mine + (int64_t)c * V::kN + k;
                *p = fmaf(d[k], xh, first ? 0.0f : *p);
                dot = fmaf(d[k] * w[k], xh, dot);
            }
        }
        const float mean = wg_sum(dot, red[turn]) / (float)H;
        for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
            float a[V::kN], d[V::kN], w[V::kN], e[V::kN];
            V::load(s[base + c], a);
            V::load(dy[base + c], d);
            V::load(weight[c], w);
            V::load(ds ? ds[base + c] : make_uint4(0, 0, 0, 0), e);
#pragma unroll
            for (int k = 0; k < V::kN; ++k)
                e[k] = fmaf(rs, fmaf(-(a[k] * rs), mean, d[k] * w[k]), e[k]);
            dx[base + c] = V::store(e);
        }
    }
}

// dweight[h] = sum over the workgroups' rows of part, in a fixed order: 16
// threads per column take every 16th row, then their sums are added in order.
__global__ __launch_bounds__(1024) void dweight_kernel(int G, int H, int h0, const float* __restrict__ part,
                                                       float* __restrict__ dweight)
{
    __shared__ float sh[16][kRedCols];
    const int col = threadIdx.x % kRedCols, grp = threadIdx.x / kRedCols;
    const int h = h0 + blockIdx.x * kRedCols + col;
    float a = 0.0f;
    if (h < H) {
        int g = grp;
        for (; g + 7 * 16 < G; g += 8 * 16) {  // eight loads in flight
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = part[(int64_t)(g + 16 * i) * H + h];
#pragma unroll
            for (int i = 0; i < 8; ++i) a += v[i];
        }
        for (; g < G; g += 16) a += part[(int64_t)g * H + h];
    }
    sh[grp][col] = a;
    __syncthreads();
    if (grp == 0 && h < H) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += sh[i][col];
        dweight[h] = t;
    }
}

// 8-bit blocks of a plain matrix: one thread per vector.
template <bool BF16>
__global__ __launch_bounds__(256) void mx_quantize_kernel(int64_t vecs, const uint4* __restrict__ x,
                                                          uint8_t* __restrict__ q,
                                                          uint8_t* __restrict__ scales)
{
    using V = Vec<BF16>;
    // whole blocks of lanes pass the end together (vecs is a multiple of
    // the lanes of a block), so the shuffles see all of a block
    for (int64_t c0 = (int64_t)blockIdx.x * 256; c0 < vecs; c0 += (int64_t)gridDim.x * 256) {
        const int64_t c = c0 + threadIdx.x;
        float f[V::kN];
        V::load(c < vecs ? x[c] : make_uint4(0, 0, 0, 0), f);
        store_mx<BF16>(f, c, c < vecs, q, scales);
    }
}

// Threads and vectors per thread for rows of `vecs` vectors: at most kMaxCh
// vectors a thread, else 0 (the wide kernels).
struct RowSplit {
    int threads, ch;
};
RowSplit row_split(int vecs)
{
    int t = vecs <= 64 ? 64 : vecs <= 128 ? 128 : 256;
    while (t < kMaxThreads && vecs > t * kMaxCh) t *= 2;
    const int ch = (vecs + t - 1) / t;
    return ch <= kMaxCh ? RowSplit{t, ch} : RowSplit{kMaxThreads, 0};
}

template <bool BF16, bool STREAM>
hipError_t launch_norm(const moe_shape_t& sh, const void* x, const void* r, const void* w, float eps,
                       void* s, void* y, void* q, void* scales, float* rstd, hipStream_t st)
{
    const int vecs = sh.H / Vec<BF16>::kN;
    const RowSplit p = row_split(vecs);
    const uint4 *xv = static_cast<const uint4*>(x), *rv = static_cast<const uint4*>(r),
                *wv = static_cast<const uint4*>(w);
    uint4 *sv = static_cast<uint4*>(s), *yv = static_cast<uint4*>(y);
    uint8_t *qv = static_cast<uint8_t*>(q), *cv = static_cast<uint8_t*>(scales);
    switch (p.ch) {
#define MOE_NORM(C)                                                                                \
    case C:                                                                                        \
        rmsnorm_kernel<BF16, C, STREAM><<<sh.T, p.threads, 0, st>>>(sh.H, vecs, xv, rv, wv, eps, sv, \
                                                                    yv, qv, cv, rstd);             \
        break;
        MOE_NORM(1) MOE_NORM(2) MOE_NORM(3) MOE_NORM(4)
#undef MOE_NORM
    default:
        rmsnorm_wide_kernel<BF16><<<sh.T, p.threads, 0, st>>>(sh.H, vecs, xv, rv, wv, eps, sv, yv, qv,
                                                              cv, rstd);
    }
    return hipGetLastError();
}

// The backward holds 7 vectors' worth of registers per vector of the row (s,
// dy, ds, the weight and the fp32 sums), so it takes two vectors a thread on
// up to 512 threads, then up to four; 12288 and 16384 columns of bf16 run at 4.9 and
// 5.0 TB/s. Past them 1024 threads have 128 registers each: enough for fp32 (12288
// columns 5.2, 16384 4.8 TB/s, the wide kernel 2.8), while bf16 spills 53 (three
// vectors) and 112 (four). Spilled / wide, 2048 rows: 20480 columns 200 / 226 us,
// 24576 219 / 279, 28672 353 / 328, 32768 372 / 381 (1.4 to 1.8 TB/s all).
template <bool BF16, bool STREAM>
hipError_t launch_norm_bwd(const moe_shape_t& sh, const void* s, const void* w, const float* rstd,
                           const void* dy, const void* ds, void* dx, float* part, int G, hipStream_t st)
{
    const int vecs = sh.H / Vec<BF16>::kN;
    const uint4 *sv = static_cast<const uint4*>(s), *wv = static_cast<const uint4*>(w),
                *dv = static_cast<const uint4*>(dy), *ev = static_cast<const uint4*>(ds);
    uint4* xv = static_cast<uint4*>(dx);
    int t = 64;
    while (t < 512 && vecs > 2 * t) t *= 2;
    if (vecs > 4 * t) t = kMaxThreads;
    const int ch = (vecs + t - 1) / t;
#define MOE_NORM(C, TH)                                                                              \
    rmsnorm_bwd_kernel<BF16, C, TH, STREAM><<<G, t, 0, st>>>(sh.T, sh.H, vecs, sv, wv, rstd, dv, ev, xv, part)
    if (t <= 512 && ch == 1) MOE_NORM(1, 512);
    else if (t <= 512 && ch == 2) MOE_NORM(2, 512);
    else if (t <= 512 && ch == 3) MOE_NORM(3, 512);
    else if (t <= 512) MOE_NORM(4, 512);
    else if (ch == 3) MOE_NORM(3, kMaxThreads);
    else if (ch == 4) MOE_NORM(4, kMaxThreads);
    else
        rmsnorm_bwd_wide_kernel<BF16><<<G, kMaxThreads, 0, st>>>(sh.T, sh.H, vecs, sv, wv, rstd, dv, ev, xv,
                                                                 part);
#undef MOE_NORM
    return hipGetLastError();
}

}  // namespace

hipError_t moe_launch_rmsnorm(const moe_shape_t& s, const void* x, const void* residual,
                              const void* weight, float eps, void* s_out, void* y, void* q,
                              void* scales, float* rstd, hipStream_t st)
{
    const int64_t row = (int64_t)s.H * (s.dtype == MOE_BF16 ? 2 : 4);
    const bool stream = s.T * (row * (1 + !!residual + !!s_out + !!y) + (q ? s.H : 0)) > moe::kStreamBytes;
    auto* launch = s.dtype == MOE_BF16 ? (stream ? launch_norm<true, true> : launch_norm<true, false>)
                                       : (stream ? launch_norm<false, true> : launch_norm<false, false>);
    // (past 2^32 threads a launch quietly runs the remainder only)
    moe_shape_t part = s;
    for (int64_t t0 = 0; t0 < s.T; t0 += kMaxRows) {
        part.T = (int)(s.T - t0 < kMaxRows ? s.T - t0 : kMaxRows);
        auto at = [&](auto* p, int64_t row_bytes) {
            using Byte = std::conditional_t<std::is_const_v<std::remove_pointer_t<decltype(p)>>, const char, char>;
            return p ? static_cast<decltype(p)>(static_cast<Byte*>(p) + t0 * row_bytes) : nullptr;
        };
        const hipError_t e = launch(part, at(x, row), at(residual, row), weight, eps, at(s_out, row), at(y, row),
                                    at(q, s.H), at(scales, s.H / moe::kMxBlock), rstd ? rstd + t0 : nullptr, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t moe_launch_rmsnorm_backward(const moe_shape_t& s, const void* s_in, const void* weight,
                                       const float* rstd, const void* dy, const void* ds, void* dx,
                                       float* dweight, float* part, hipStream_t st)
{
    const int G = moe::norm_bwd_groups(s);
    if (G > 0) {
        const int64_t row = (int64_t)s.H * (s.dtype == MOE_BF16 ? 2 : 4);
        const bool stream = s.T * row * (3 + !!ds) > moe::kStreamBytes;
        auto* launch = s.dtype == MOE_BF16 ? (stream ? launch_norm_bwd<true, true> : launch_norm_bwd<true, false>)
                                           : (stream ? launch_norm_bwd<false, true> : launch_norm_bwd<false, false>);
        const hipError_t e = launch(s, s_in, weight, rstd, dy, ds, dx, part, G, st);
        if (e != hipSuccess) return e;
    }
    for (int64_t h0 = 0; h0 < s.H; h0 += (int64_t)kMaxRows * kRedCols) {
        const int64_t left = (s.H - h0 + kRedCols - 1) / kRedCols;
        dweight_kernel<<<(int)(left < kMaxRows ? left : kMaxRows), 1024, 0, st>>>(G, s.H, (int)h0, part, dweight);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t moe_launch_mx_quantize(int64_t rows, int64_t cols, int dtype, const void* x, void* q,
                                  void* scales, hipStream_t st)
{
    if (rows == 0) return hipSuccess;
    const bool bf = dtype == MOE_BF16;
    const int64_t vecs = rows * cols / (bf ? 8 : 4);
    const int64_t want = (vecs + 255) / 256;
    const int grid = (int)(want < 16384 ? want : 16384);
    const uint4* xv = static_cast<const uint4*>(x);
    uint8_t *qv = static_cast<uint8_t*>(q), *sv = static_cast<uint8_t*>(scales);
    if (bf) mx_quantize_kernel<true><<<grid, 256, 0, st>>>(vecs, xv, qv, sv);
    else mx_quantize_kernel<false><<<grid, 256, 0, st>>>(vecs, xv, qv, sv);
    return hipGetLastError();
}
