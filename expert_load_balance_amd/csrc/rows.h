// rows.h -- rows of values in the layer's types: 16-byte vectors, sums over a
// workgroup, 8-bit blocks (the norms' kernels).
#pragma once

#include "mx.h"

namespace moe {
namespace rows {

template <bool BF16>
struct Vec;
template <>
struct Vec<true> {
    static constexpr int kN = 8;
    __device__ static void load(const uint4& u, float* f)
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 store(const float* f)
    {
        return make_uint4(moe::pack_bf16x2(f[0], f[1]), moe::pack_bf16x2(f[2], f[3]),
                          moe::pack_bf16x2(f[4], f[5]), moe::pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Vec<false> {
    static constexpr int kN = 4;
    __device__ static void load(const uint4& u, float* f)
    {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    __device__ static uint4 store(const float* f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};

// Sum over the workgroup; every thread gets it. red: 16 values of LDS no
// other call of the same row uses.
template <typename T>
__device__ __forceinline__ T wg_sum(T v, T* red)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
    const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    T t = 0;
    for (int i = 0; i < waves; ++i) t += red[i];
    return t;
}

// rstd from the sum of squares, in fp64 like the sum: rstd is then the
// correctly rounded one but for a tie, and a code or a bf16 of v goes to the
// other side of a rounding only by the two fp32 products. The memory traffic
// hides the fp64 adds (one conversion and one multiply-add per element).
__device__ __forceinline__ float rstd_of(double ss, int H, float eps)
{
    return (float)(1.0 / sqrt(ss / (double)H + (double)eps));
}

// One vector of v to q and scales: 32 columns are 4 (bf16) or 8 (fp32)
// neighbouring lanes, which hold the whole block (H % 32 == 0; the lanes past
// the row are whole blocks too and store nothing).
template <bool BF16>
__device__ __forceinline__ void store_mx(const float* v, int64_t vec, bool in, uint8_t* q, uint8_t* scales)
{
    constexpr int N = Vec<BF16>::kN, kLanes = moe::kMxBlock / N;
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) top = max(top, moe::mx_mag(v[k]));
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    const uint32_t byte = moe::mx_scale_byte(top);
    uint32_t w[N / 4];
#pragma unroll
    for (int k = 0; k < N / 4; ++k)
        w[k] = moe::mx_pack4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], byte);
    if (!in) return;
    if (BF16) *reinterpret_cast<uint2*>(q + vec * 8) = make_uint2(w[0], w[N / 4 - 1]);
    else *reinterpret_cast<uint32_t*>(q + vec * 4) = w[0];
    if ((threadIdx.x & (kLanes - 1)) == 0) scales[vec / kLanes] = (uint8_t)byte;
}

}  // namespace rows
}  // namespace moe
