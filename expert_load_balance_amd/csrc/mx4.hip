// mx4.hip -- 4-bit blocks of a matrix, and their values back.
//
// Bound by memory. A thread takes eight values: 16 bytes of bf16 (or 32 of
// fp32) against 4 bytes of codes, so that a wave reads and writes whole lines;
// four neighbouring lanes hold a block. It has four such eights in flight: 805 M
// bf16 values 323 us (2.04 GB, 6.3 TB/s), back 352 (5.8 TB/s); eight of them took
// 331 and 361, and matrices of this size read and written through the caches 399. 403 M
// fp32 values 342 us (5.3 TB/s), back 454 (4.0 TB/s).
#include "lanes.h"
#include "rows.h"
#include "step.h"

namespace {

using moe::rows::Vec;

constexpr int kThreads = 256, kEach = 4;  // eights of a thread at a time
constexpr int kMaxGrid = 16384;

// An eight of values in 16-byte vectors.
template <bool BF16>
struct Eight {
    uint4 v[BF16 ? 1 : 2];
    template <bool STREAM>
    __device__ void load(const uint4* x, int64_t i)
    {
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k) v[k] = moe::load16<STREAM>(x + (BF16 ? 1 : 2) * i + k);
    }
    __device__ void values(float* f) const
    {
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k) Vec<BF16>::load(v[k], f + 4 * k);
    }
    template <bool STREAM>
    __device__ static void store(uint4* x, int64_t i, const float* f)
    {
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k)
            moe::store16<STREAM>(x + (BF16 ? 1 : 2) * i + k, Vec<BF16>::store(f + 4 * k));
    }
};

// n: eights of values, a multiple of four, so that the lanes of a block pass the end
// together and the shuffles see all of it
template <bool BF16, bool STREAM>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(int64_t n, const uint4* __restrict__ x,
                                                                uint32_t* __restrict__ q,
                                                                uint8_t* __restrict__ scales)
{
    for (int64_t at = (int64_t)blockIdx.x * (kThreads * kEach); at < n; at += (int64_t)gridDim.x * (kThreads * kEach)) {
        Eight<BF16> e[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int64_t i = at + u * kThreads + threadIdx.x;
            if (i < n) e[u].template load<STREAM>(x, i);
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int64_t i = at + u * kThreads + threadIdx.x;
            if (i >= n) continue;
            float f[8];
            e[u].values(f);
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, moe::mx_mag(f[k]));
            top = max(top, (uint32_t)moe::lanes::dpp<moe::lanes::kQuadXor1>((int)top));
            top = max(top, (uint32_t)moe::lanes::dpp<moe::lanes::kQuadXor2>((int)top));
            const uint32_t byte = moe::mx4_scale_byte(top);
            const uint32_t codes = moe::mx4_pack8(f, byte);
            if (STREAM) __builtin_nontemporal_store(codes, q + i);
            else q[i] = codes;
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
        }
    }
}

template <bool BF16, bool STREAM>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(int64_t n, const uint32_t* __restrict__ q,
                                                                  const uint8_t* __restrict__ scales,
                                                                  uint4* __restrict__ x)
{
    for (int64_t at = (int64_t)blockIdx.x * (kThreads * kEach); at < n; at += (int64_t)gridDim.x * (kThreads * kEach)) {
        uint32_t c[kEach], s[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int64_t i = at + u * kThreads + threadIdx.x;
            c[u] = i < n ? STREAM ? __builtin_nontemporal_load(q + i) : q[i] : 0u;
            s[u] = i < n ? scales[i >> 2] : 0u;
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int64_t i = at + u * kThreads + threadIdx.x;
            float f[8];
            moe::mx4_unpack8(c[u], moe::mx_scale_value(s[u]), f);
            if (i < n) Eight<BF16>::template store<STREAM>(x, i, f);
        }
    }
}

int grid_of(int64_t n)
{
    const int64_t want = (n + kThreads * kEach - 1) / (kThreads * kEach);
    return (int)(want < kMaxGrid ? want : kMaxGrid);
}
// Whether a call's values are more than the caches hold (see mx.h).
bool past_caches(int64_t n, int dtype) { return n * (dtype == MOE_BF16 ? 16 : 32) > moe::kStreamBytes; }

}  // namespace

hipError_t moe_launch_mx4_quantize(int64_t rows, int64_t cols, int dtype, const void* x, void* q, void* scales,
                                   hipStream_t st)
{
    if (rows == 0) return hipSuccess;
    const int64_t n = rows * cols / 8;
    const uint4* xv = static_cast<const uint4*>(x);
    uint32_t* qv = static_cast<uint32_t*>(q);
    uint8_t* sv = static_cast<uint8_t*>(scales);
    const bool bf = dtype == MOE_BF16;
    auto* kernel = past_caches(n, dtype) ? (bf ? mx4_quantize_kernel<true, true> : mx4_quantize_kernel<false, true>)
                                         : (bf ? mx4_quantize_kernel<true, false> : mx4_quantize_kernel<false, false>);
    kernel<<<grid_of(n), kThreads, 0, st>>>(n, xv, qv, sv);
    return hipGetLastError();
}

hipError_t moe_launch_mx4_dequantize(int64_t rows, int64_t cols, int dtype, const void* q, const void* scales, void* x,
                                     hipStream_t st)
{
    if (rows == 0) return hipSuccess;
    const int64_t n = rows * cols / 8;
    const uint32_t* qv = static_cast<const uint32_t*>(q);
    const uint8_t* sv = static_cast<const uint8_t*>(scales);
    uint4* xv = static_cast<uint4*>(x);
    const bool bf = dtype == MOE_BF16;
    auto* kernel = past_caches(n, dtype) ? (bf ? mx4_dequantize_kernel<true, true> : mx4_dequantize_kernel<false, true>)
                                         : (bf ? mx4_dequantize_kernel<true, false> : mx4_dequantize_kernel<false, false>);
    kernel<<<grid_of(n), kThreads, 0, st>>>(n, qv, sv, xv);
    return hipGetLastError();
}
