// lanes.h -- reductions across the lanes of a wavefront without LDS (gfx950).
#pragma once

#include "common.h"

namespace moe {
namespace lanes {

// Cross-lane steps without LDS: DPP moves inside rows of 16 lanes and the
// gfx950 permlane swaps across rows. For an all-reduce of a commutative op a
// partner from the other half of the current group is enough, so the
// mirrors stand in for xor 4 and xor 8 once the smaller groups are reduced.
constexpr int kQuadXor1 = 0xB1;     // quad_perm [1,0,3,2]
constexpr int kQuadXor2 = 0x4E;     // quad_perm [2,3,0,1]
constexpr int kHalfMirror = 0x141;  // lane i <-> 7-i in each 8
constexpr int kMirror = 0x140;      // lane i <-> 15-i in each 16

template <int CTRL>
__device__ __forceinline__ int dpp(int v)
{
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, v)));
}

// A copy the optimiser cannot see through. The permlane swaps below take the
// same value as both operands; the compiler was seen to treat the second
// half of such a swap as equal to the first and drop it, so each swap gets
// an opaque copy as its second operand.
__device__ __forceinline__ int opaque(int v)
{
    int r;
    asm volatile("v_mov_b32 %0, %1" : "=v"(r) : "v"(v));
    return r;
}

// the rows of 16 (ROWS32 false) or 32 lanes paired by a permlane swap: every
// lane gets {its own row's value, the paired row's value} in row order
template <bool ROWS32>
__device__ __forceinline__ void swap_halves(int v, int& lo, int& hi)
{
    if constexpr (ROWS32) {
        const auto s = __builtin_amdgcn_permlane32_swap(v, opaque(v), false, false);
        lo = (int)s[0];
        hi = (int)s[1];
    } else {
        const auto s = __builtin_amdgcn_permlane16_swap(v, opaque(v), false, false);
        lo = (int)s[0];
        hi = (int)s[1];
    }
}

template <bool SUM>
__device__ __forceinline__ float op(float a, float b)
{
    return SUM ? a + b : fmaxf(a, b);
}

template <bool SUM, bool ROWS32>
__device__ __forceinline__ float swap_op(float x)
{
    int lo, hi;
    swap_halves<ROWS32>(__builtin_bit_cast(int, x), lo, hi);
    return op<SUM>(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}

// max or sum over a group; every lane gets the same value (each step is commutative)
template <int G, bool SUM>
__device__ __forceinline__ float group_reduce(float v)
{
    if constexpr (G >= 2) v = op<SUM>(v, dpp<kQuadXor1>(v));
    if constexpr (G >= 4) v = op<SUM>(v, dpp<kQuadXor2>(v));
    if constexpr (G >= 8) v = op<SUM>(v, dpp<kHalfMirror>(v));
    if constexpr (G >= 16) v = op<SUM>(v, dpp<kMirror>(v));
    if constexpr (G >= 32) v = swap_op<SUM, false>(v);
    if constexpr (G >= 64) v = swap_op<SUM, true>(v);
    return v;
}

}  // namespace lanes
}  // namespace moe
