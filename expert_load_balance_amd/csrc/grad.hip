// grad.hip -- the global norm of a list of gradients, and clipping to it.
//
//   norm = sqrt(sum g^2), dst = src * (max / norm if norm > max else 1).
//
// Bound by memory: one read for the norm, one read and one write for the
// clip. The tensors are cut into chunks of kChunk elements, and the chunks
// of all tensors (up to kMaxTensors per launch, passed by value, so a captured
// call holds its list) are dealt to the workgroups in turn. The squares are
// added in fp64: no overflow or lost small values whatever the gradients'
// range, and the adds cost less than the loads (one conversion and one
// multiply-add per element).
//
// Measured: 1.4 billion fp32 values, norm 838 us (6.7 TB/s), clip 2215 us (5.1
// TB/s read + written; the same in place), through the caches 970 and 2255; 96 tensors
// of 164 MB in bf16 and fp32, 27 + 4 and 58 us in one launch each, 84 us both from a
// graph, 98 in place; the rest of the out-of-place call's 130 us is the host's, which
// walks the list of gradients for each call and the outputs' for the second. The
// clip's pass over what the norm has just read in reverse order (for what the caches
// still hold) changed nothing.
//
// A tensor that does not start on 16 bytes is read and written an element at a
// time: 400 million values one element off, norm and clip, bf16 678 and 572 us (aligned
// 121 and 277), fp32 741 and 756 us (237 and 612).
#include <math.h>

#include "mx.h"

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;       // elements per chunk
constexpr int kMaxTensors = 96;     // per launch: 2.8 KB of the 4 KB of kernel arguments
constexpr int kGroups = 2048;       // most workgroups of one launch

struct Batch {
    const void* src[kMaxTensors];
    void* dst[kMaxTensors];
    int64_t count[kMaxTensors];
    int32_t start[kMaxTensors + 1]; // first chunk of each tensor
    uint8_t bf16[kMaxTensors];
    int32_t n;
};

// The tensor that holds chunk c (chunks of empty tensors do not exist).
__device__ __forceinline__ int tensor_of(const Batch& b, int c)
{
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.start[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ void add_sq(double& a, float f)
{
    const double d = (double)f;
    a = fma(d, d, a);
}

__device__ __forceinline__ bool aligned16(const void* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <bool STREAM>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const Batch b, int chunks,
                                                             double* __restrict__ part)
{
    double a0 = 0.0, a1 = 0.0, a2 = 0.0, a3 = 0.0;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of(b, c);
        const int64_t e0 = (int64_t)(c - b.start[t]) * kChunk;
        const int64_t left = b.count[t] - e0;
        const int n = (int)(left < kChunk ? left : kChunk);
        if (b.bf16[t]) {
            const uint16_t* p = static_cast<const uint16_t*>(b.src[t]) + e0;
            int i0 = 0;
            if (aligned16(p)) {
                i0 = n / 8 * 8;
                const uint4* v = reinterpret_cast<const uint4*>(p);
#pragma unroll 4
                for (int i = threadIdx.x; i < n / 8; i += kThreads) {
                    const uint4 u = moe::load16<STREAM>(v + i);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        add_sq(k & 1 ? a2 : a0, __uint_as_float(w[k] << 16));
                        add_sq(k & 1 ? a3 : a1, __uint_as_float(w[k] & 0xffff0000u));
                    }
                }
            }
            for (int i = i0 + threadIdx.x; i < n; i += kThreads) add_sq(a0, moe::bf16_bits_to_f32(p[i]));
        } else {
            const float* p = static_cast<const float*>(b.src[t]) + e0;
            int i0 = 0;
            if (aligned16(p)) {
                i0 = n / 4 * 4;
                const uint4* v = reinterpret_cast<const uint4*>(p);
#pragma unroll 4
                for (int i = threadIdx.x; i < n / 4; i += kThreads) {
                    const uint4 u = moe::load16<STREAM>(v + i);
                    add_sq(a0, __uint_as_float(u.x));
                    add_sq(a1, __uint_as_float(u.y));
                    add_sq(a2, __uint_as_float(u.z));
                    add_sq(a3, __uint_as_float(u.w));
                }
            }
            for (int i = i0 + threadIdx.x; i < n; i += kThreads) add_sq(a0, p[i]);
        }
    }
    double a = (a0 + a1) + (a2 + a3);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) a += __shfl_xor(a, off);
    __shared__ double red[kThreads / 64];
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    if (threadIdx.x == 0) part[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(1024) void grad_total_kernel(int64_t n, const double* __restrict__ part,
                                                          float* __restrict__ norm, int32_t* err)
{
    __shared__ double red[16];
    double a = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) a += part[i];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) a += __shfl_xor(a, off);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int i = 0; i < 16; ++i) t += red[i];
        const float r = (float)sqrt(t);
        *norm = r;
        if (!(r < __uint_as_float(0x7f800000u))) atomicOr(err, MOE_ERR_NONFINITE);
    }
}

// src may be dst
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(const Batch b, int chunks, float max_norm,
                                                             const float* __restrict__ norm)
{
    const float r = *norm;
    const bool over = r > max_norm && r < __uint_as_float(0x7f800000u);
    const float s = over ? (float)((double)max_norm / (double)r) : 1.0f;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of(b, c);
        if (!over && b.src[t] == b.dst[t]) continue;
        const int64_t e0 = (int64_t)(c - b.start[t]) * kChunk;
        const int64_t left = b.count[t] - e0;
        const int n = (int)(left < kChunk ? left : kChunk);
        if (b.bf16[t]) {
            const uint16_t* p = static_cast<const uint16_t*>(b.src[t]) + e0;
            uint16_t* o = static_cast<uint16_t*>(b.dst[t]) + e0;
            int i0 = 0;
            if (aligned16(p) && aligned16(o)) {
                i0 = n / 8 * 8;
#pragma unroll 4
                for (int i = threadIdx.x; i < n / 8; i += kThreads) {
                    uint4 u = moe::load16<STREAM>(reinterpret_cast<const uint4*>(p) + i);
                    uint32_t* w = &u.x;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = moe::pack_bf16x2(__uint_as_float(w[k] << 16) * s,
                                                __uint_as_float(w[k] & 0xffff0000u) * s);
                    moe::store16<STREAM>(reinterpret_cast<uint4*>(o) + i, u);
                }
            }
            for (int i = i0 + threadIdx.x; i < n; i += kThreads)
                o[i] = moe::f32_to_bf16_bits(moe::bf16_bits_to_f32(p[i]) * s);
        } else {
            const float* p = static_cast<const float*>(b.src[t]) + e0;
            float* o = static_cast<float*>(b.dst[t]) + e0;
            int i0 = 0;
            if (aligned16(p) && aligned16(o)) {
                i0 = n / 4 * 4;
#pragma unroll 4
                for (int i = threadIdx.x; i < n / 4; i += kThreads) {
                    uint4 u = moe::load16<STREAM>(reinterpret_cast<const uint4*>(p) + i);
                    uint32_t* w = &u.x;
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * s);
                    moe::store16<STREAM>(reinterpret_cast<uint4*>(o) + i, u);
                }
            }
            for (int i = i0 + threadIdx.x; i < n; i += kThreads) o[i] = p[i] * s;
        }
    }
}

// Calls f(batch, chunks, groups, first partial) for each launch's share of
// the list: up to kMaxTensors tensors that are not empty, and fewer than 2^31 chunks.
template <typename F>
hipError_t for_batches(int n, const moe_grad_t* g, F f)
{
    int64_t first = 0;
    for (int i = 0; i < n;) {
        Batch b;
        b.n = 0;
        int64_t chunks = 0;
        for (; i < n && b.n < kMaxTensors; ++i) {
            const int64_t c = (g[i].count + kChunk - 1) / kChunk;
            if (c == 0) continue;
            if (chunks + c >= (int64_t(1) << 31)) break;  // one tensor has at most 2^26 chunks
            b.src[b.n] = g[i].src;
            b.dst[b.n] = g[i].dst;
            b.count[b.n] = g[i].count;
            b.start[b.n] = (int32_t)chunks;
            b.bf16[b.n] = g[i].dtype == MOE_BF16;
            chunks += c;
            ++b.n;
        }
        if (b.n == 0) continue;
        b.start[b.n] = (int32_t)chunks;
        const int groups = chunks < kGroups ? (int)chunks : kGroups;
        const hipError_t e = f(b, (int)chunks, groups, first);
        if (e != hipSuccess) return e;
        first += groups;
    }
    return hipSuccess;
}

// Whether the list is past what the caches keep from the norm to the clip.
bool streamed(int n, const moe_grad_t* g)
{
    int64_t bytes = 0;
    for (int i = 0; i < n && bytes <= moe::kStreamBytes; ++i) bytes += g[i].count * (g[i].dtype == MOE_BF16 ? 2 : 4);
    return bytes > moe::kStreamBytes;
}

int64_t partials(int n, const moe_grad_t* g)
{
    int64_t total = 0;
    (void)for_batches(n, g, [&](const Batch&, int, int groups, int64_t first) {
        total = first + groups;
        return hipSuccess;
    });
    return total;
}

}  // namespace

size_t moe_grad_ws_bytes(int n, const moe_grad_t* g)
{
    const int64_t p = partials(n, g);
    return moe::align256((size_t)(p > 0 ? p : 1) * sizeof(double));
}

hipError_t moe_launch_grad_norm(int n, const moe_grad_t* g, float* norm, int32_t* err, double* part,
                                hipStream_t st)
{
    int64_t total = 0;
    auto* kernel = streamed(n, g) ? grad_norm_kernel<true> : grad_norm_kernel<false>;
    const hipError_t e = for_batches(n, g, [&](const Batch& b, int chunks, int groups, int64_t first) {
        kernel<<<groups, kThreads, 0, st>>>(b, chunks, part + first);
        total = first + groups;
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    grad_total_kernel<<<1, 1024, 0, st>>>(total, part, norm, err);
    return hipGetLastError();
}

hipError_t moe_launch_grad_clip(int n, const moe_grad_t* g, float max_norm, const float* norm,
                                hipStream_t st)
{
    auto* kernel = streamed(n, g) ? grad_clip_kernel<true> : grad_clip_kernel<false>;
    return for_batches(n, g, [&](const Batch& b, int chunks, int groups, int64_t) {
        kernel<<<groups, kThreads, 0, st>>>(b, chunks, max_norm, norm);
        return hipGetLastError();
    });
}
