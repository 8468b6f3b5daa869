// step.h -- 4-bit blocks on gfx950, sizes of the operators of moe_step.h, and
// their launchers.
#pragma once

#include "moe_step.h"
#include "mx.h"

namespace moe {

// Scale byte of a 4-bit block whose largest magnitude has the bits `top`: the
// smallest e >= -127 with top <= 6 * 2^e = 1.5 * 2^(e + 2), as e + 127. With
// top = m * 2^x, m in [1, 2), e is x - 2 where m <= 1.5, else x - 1: adding
// 0x3fffff carries into the exponent exactly when the mantissa field exceeds
// 0x400000. Infinities and NaN give 255.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t top)
{
    const int e = (int)((top + 0x3fffffu) >> 23) - 2;
    return top >= 0x7f800000u ? 255u : (uint32_t)(e > 0 ? e : 0);
}

// Eight e2m1 codes of values divided by the block's scale, first in the low
// half of the low byte (the quotients are at most 6, the conversion is to
// nearest even). A scale byte of 255 has codes of 0.
__device__ __forceinline__ uint32_t mx4_pack8(const float* v, uint32_t byte)
{
    const float s = __uint_as_float(byte << 23);  // (taken by its exponent: 0 is 2^-127)
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
    return byte == 255u ? 0u : r;
}

// A scale byte's value: 2^-127 is a subnormal, 255 is NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t byte)
{
    return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}

// Eight values of e2m1 codes times s.
__device__ __forceinline__ void mx4_unpack8(uint32_t codes, float s, float* v)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
    v[0] = a[0] * s, v[1] = a[1] * s, v[2] = b[0] * s, v[3] = b[1] * s;
    v[4] = c[0] * s, v[5] = c[1] * s, v[6] = d[0] * s, v[7] = d[1] * s;
}

// Rows of the backward of moe_block_norm in parts: of the rows that share a row of
// gates a part takes every per_group-th, so that the rows in work at one time are
// neighbours. As many workgroups as fit on the chip at once (16 waves a CU; or as
// many as there are parts) take parts b, b + G, ... 8192 rows of 7168 bf16, one
// gate a channel: 131 us on 256 workgroups, 143 on 512, 152 on 768.
inline int block_norm_groups(const moe_shape_t& s)
{
    const int waves = (s.H / (s.dtype == MOE_BF16 ? 8 : 4) + 63) / 64;
    return kGemmMaxGrid * (waves > 8 ? 1 : waves > 4 ? 2 : 4);
}
struct BlockNormParts {
    int64_t group_rows, groups;  // rows that share a row of gates, and how many such groups
    int per_group;               // parts of a group
    int64_t parts;
    int grid;
};
inline BlockNormParts block_norm_parts(const moe_shape_t& s, int32_t gate_rows)
{
    const int64_t T = s.T, G = block_norm_groups(s);
    BlockNormParts p;
    p.group_rows = gate_rows > 0 && gate_rows < T ? gate_rows : T > 0 ? T : 1;
    p.groups = (T + p.group_rows - 1) / p.group_rows;
    const int64_t n = p.groups > 0 ? (G + p.groups - 1) / p.groups : 1;
    p.per_group = (int)(n < p.group_rows ? n : p.group_rows);
    p.parts = p.groups * p.per_group;
    p.grid = (int)(p.parts < G ? p.parts : G);
    return p;
}
// Workspace: dw_post and dw_pre of each workgroup, then, where groups have
// several parts, the gate's gradient of each part (fp32 [H] each).
inline size_t block_norm_bwd_ws(const moe_shape_t& s, int32_t gate_rows)
{
    const BlockNormParts p = block_norm_parts(s, gate_rows);
    const size_t rows = 2 * (size_t)(p.grid > 0 ? p.grid : 1) +
                        (gate_rows > 0 && p.per_group > 1 ? (size_t)p.parts : 0);
    return align256(rows * s.H * 4);
}

}  // namespace moe

struct MoeBlockNorm {
    const void *x, *residual;
    float alpha;
    const void *w_post, *gate;
    int gate_rows;
    const void* w_pre;
    float eps;
    void *s, *y, *q, *scales;
    float *rstd_post, *rstd_pre;
};
struct MoeBlockNormBwd {
    const void* x;
    const float* rstd_post;
    const void* s;
    const float* rstd_pre;
    float alpha;
    const void *w_post, *gate;
    int gate_rows;
    const void *w_pre, *dy, *ds;
    void *dx, *dresidual;
    float *dw_post, *dgate, *dw_pre;
};
hipError_t moe_launch_block_norm(const moe_shape_t& s, const MoeBlockNorm& a, hipStream_t st);
hipError_t moe_launch_block_norm_backward(const moe_shape_t& s, const MoeBlockNormBwd& a, float* ws,
                                          hipStream_t st);
hipError_t moe_launch_mx4_quantize(int64_t rows, int64_t cols, int dtype, const void* x, void* q,
                                   void* scales, hipStream_t st);
hipError_t moe_launch_mx4_dequantize(int64_t rows, int64_t cols, int dtype, const void* q,
                                     const void* scales, void* x, hipStream_t st);
hipError_t moe_launch_grouped_gemm_mx4(const moe_shape_t& s, const void* a, const void* a_s,
                                       const int32_t* plan, const MoeMxWeights& w, void* y,
                                       char* ws, hipStream_t st);

// --------------------------------------------- the layer for a few tokens --
namespace moe {

constexpr int kFewMaxH = 8192;   // a wave's part of a row of x stays in registers
constexpr int kFewPart = 4096;   // values of K of a part of the down projection (h in registers, two bf16 each)
constexpr int kFewTile = 16;     // rows of a tile

constexpr int kFewTableBytes = 8192; // rows and entries of the choice, at most
constexpr int kFewLogitK = 1024; // values of H of a part of the router's scores
constexpr int kFewLogitParts = kFewMaxH / kFewLogitK;

inline int few_logit_parts(int H) { return (H + kFewLogitK - 1) / kFewLogitK; }
inline int few_unit(int form) { return form == MOE_W_BF16 ? 64 : 128; }
// Whether an expert's rows may be two tiles, so that its weights are read once: where
// experts have more than 8 rows on average. (Two tiles' h takes parts of half the
// length. us, one tile and two: 4 experts, all chosen by 17 tokens, 4096 x 14336, 8-bit 248
// and 161; 4-bit, top-8 of 16, 4096 x 4096, 17 tokens (8.5 rows) 99.5 and 100.7, 24
// tokens 125 and 105 to 117; 4-bit, top-2 of 8, 4096 x 14336, 32 tokens (8 rows) 151 and 162.)
inline bool few_two_tiles(const moe_shape_t& s) { return s.T > kFewTile && s.T * s.k > 8 * s.E; }
inline int few_parts(int F, bool two_tiles)
{
    const int part = two_tiles ? kFewPart / 2 : kFewPart;
    return (F + part - 1) / part;
}

// logits [parts][T][E], the router's w [N], each assignment's row [N], the choice's tables, h in two bf16
// planes [N][F] + [T][shared_F], y fp32 [parts][N][H] + [shared parts][T][H]
struct FewWsLayout {
    size_t logits, w, row_of, tables, h, y, total;
    size_t h_shared, h_plane;   // elements: where the shared expert's rows begin, and the second plane
    size_t y_shared;            // elements
};
inline FewWsLayout few_ws_layout(const moe_shape_t& s, int shared_F)
{
    const size_t N = (size_t)s.T * s.k, n1 = N > 0 ? N : 1;
    FewWsLayout w;
    size_t o = 0;
    w.logits = o; o = align256(o + ((size_t)few_logit_parts(s.H) * s.T * s.E + 1) * 4);
    w.w = o;      o = align256(o + n1 * 4);
    w.row_of = o; o = align256(o + n1 * 4);
    w.tables = o; o = align256(o + kFewTableBytes);
    w.h_shared = N * s.F;
    w.h_plane = w.h_shared + (size_t)s.T * shared_F;
    w.h = o;      o = align256(o + 2 * w.h_plane * 2);
    w.y_shared = (size_t)few_parts(s.F, few_two_tiles(s)) * N * s.H;
    w.y = o;      o = align256(o + (w.y_shared + (size_t)few_parts(shared_F, few_two_tiles(s)) * s.T * s.H) * 4);
    w.total = o;
    return w;
}

}  // namespace moe

struct MoeFew {
    const void *x, *w_router;
    const float* bias;
    moe_few_weights_t routed, shared;
    int form, shared_F;
    void* out;
    int32_t* ids;
    float* w;
    int32_t* err;
};
hipError_t moe_launch_few(const moe_shape_t& s, const MoeFew& a, char* ws, hipStream_t st);
