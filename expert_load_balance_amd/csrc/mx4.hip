// mx4.hip -- 4-bit blocks of a matrix, and their values back.
//
// Bound by memory. A thread takes eight values: 16 bytes of bf16 (or 32 of
// fp32) against 4 bytes of codes, so that a wave reads and writes whole lines;
// four neighbouring lanes hold a block.
#include "rows.h"
#include "step.h"

namespace {

using moe::rows::Vec;

constexpr int kThreads = 256;
constexpr int kMaxGrid = 16384;

template <bool BF16>
__device__ __forceinline__ void load8(const uint4* x, int64_t i, float* f)
{
    if (BF16) {
        Vec<true>::load(x[i], f);
    } else {
        Vec<false>::load(x[2 * i], f);
        Vec<false>::load(x[2 * i + 1], f + 4);
    }
}
template <bool BF16>
__device__ __forceinline__ void store8(uint4* x, int64_t i, const float* f)
{
    if (BF16) {
        x[i] = Vec<true>::store(f);
    } else {
        x[2 * i] = Vec<false>::store(f);
        x[2 * i + 1] = Vec<false>::store(f + 4);
    }
}

// n: eights of values, a multiple of four
template <bool BF16>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(int64_t n, const uint4* __restrict__ x,
                                                                uint32_t* __restrict__ q,
                                                                uint8_t* __restrict__ scales)
{
    // (a block's lanes pass the end together, so the shuffles see all of it)
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        float f[8];
        load8<BF16>(x, i, f);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, moe::mx_mag(f[k]));
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const uint32_t byte = moe::mx4_scale_byte(top);
        q[i] = moe::mx4_pack8(f, byte);
        if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(int64_t n, const uint32_t* __restrict__ q,
                                                                  const uint8_t* __restrict__ scales,
                                                                  uint4* __restrict__ x)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        float f[8];
        moe::mx4_unpack8(q[i], moe::mx_scale_value(scales[i >> 2]), f);
        store8<BF16>(x, i, f);
    }
}

int grid_of(int64_t n)
{
    const int64_t want = (n + kThreads - 1) / kThreads;
    return (int)(want < kMaxGrid ? want : kMaxGrid);
}

}  // namespace

hipError_t moe_launch_mx4_quantize(int64_t rows, int64_t cols, int dtype, const void* x, void* q, void* scales,
                                   hipStream_t st)
{
    if (rows == 0) return hipSuccess;
    const int64_t n = rows * cols / 8;
    const uint4* xv = static_cast<const uint4*>(x);
    uint32_t* qv = static_cast<uint32_t*>(q);
    uint8_t* sv = static_cast<uint8_t*>(scales);
    if (dtype == MOE_BF16) mx4_quantize_kernel<true><<<grid_of(n), kThreads, 0, st>>>(n, xv, qv, sv);
    else mx4_quantize_kernel<false><<<grid_of(n), kThreads, 0, st>>>(n, xv, qv, sv);
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
    if (dtype == MOE_BF16) mx4_dequantize_kernel<true><<<grid_of(n), kThreads, 0, st>>>(n, qv, sv, xv);
    else mx4_dequantize_kernel<false><<<grid_of(n), kThreads, 0, st>>>(n, qv, sv, xv);
    return hipGetLastError();
}
