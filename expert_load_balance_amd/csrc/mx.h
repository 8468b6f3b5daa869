// mx.h -- 8-bit blocks on gfx950: 32 values of a row share a power-of-two
// scale (byte e + 127), codes are e4m3. Also the workspace of the 8-bit
// grouped GEMM and the launchers of the operators around the layer.
#pragma once

#include "common.h"
#include "moe_block.h"

namespace moe {

constexpr int kMxBlock = 32;

// Scale byte of a block whose largest magnitude has the bits `top`: the
// smallest e >= -127 with top <= 448 * 2^e = 1.75 * 2^(e + 8), as e + 127.
// With top = m * 2^x, m in [1, 2), e is x - 8 where m <= 1.75, else x - 7:
// adding 0x1fffff to the bits carries into the exponent exactly when the
// mantissa field exceeds 0x600000 (m > 1.75). Infinities and NaN give 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top)
{
    const int e = (int)((top + 0x1fffffu) >> 23) - 8;
    return top >= 0x7f800000u ? 255u : (uint32_t)(e > 0 ? e : 0);
}

// Four e4m3 codes of values divided by the block's scale (its byte as an
// exponent; the division is exact), first in the low byte. The quotients are
// at most 448 in magnitude, so the conversion (to nearest even) never
// saturates; a scale byte of 255 makes every code NaN.
__device__ __forceinline__ uint32_t mx_pack4(float a, float b, float c, float d, uint32_t byte)
{
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(byte << 23);
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, s, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, s, true);
    return __builtin_bit_cast(uint32_t, r);
}

// Bits of |v|, for a block maximum taken over unsigned integers: they order
// as the magnitudes do, infinities above every number and NaN above those.
__device__ __forceinline__ uint32_t mx_mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Calls that move more than the Infinity Cache holds (256 MB) read and write
// past the caches (non-temporal): what they leave there serves no one, and the
// dirty lines they push out cost bandwidth. Smaller ones leave their outputs for
// the next kernel. Measured on a chain of a kernel that writes x, the norm, and
// one that reads y, in us (kept / streamed), by the norm's bytes: forward 153 MB
// 43 / 49, 229 MB 70 / 69, 305 MB 90 / 90, 534 MB 169 / 162; backward 46 / 48, 67 /
// 68, 87 / 85, 170 / 152.
constexpr int64_t kStreamBytes = int64_t(256) << 20;

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint4* p)
{
    if (!STREAM) return *p;
    const u32x4v v = __builtin_nontemporal_load(reinterpret_cast<const u32x4v*>(p));
    return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool STREAM>
__device__ __forceinline__ void store16(uint4* p, const uint4& v)
{
    if (!STREAM) *p = v;
    else __builtin_nontemporal_store(u32x4v{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4v*>(p));
}

// 8-bit GEMM geometry: a workgroup tile is 256, 128, 64 or 32 rows (kinds 0..3)
// x 256 weight rows (gate/up: 128 of each), K in stages of 128 bytes (four
// scale blocks), on at most kGemmMaxGrid persistent workgroups.
constexpr int kMxTileN = 256;
constexpr int kMxStage = 128;
constexpr int kMxKinds = 4;
constexpr int kMxMinStages = 4;  // of a K-part
__host__ __device__ constexpr int mx_rows(int kind) { return 256 >> kind; }

// Kind of an expert's whole tiles: the 256-row kernel reads its scales 16
// bytes (512 values of K) at a time. One schedule serves both projections, so the
// shorter K decides for both.
__host__ inline int mx_base(const moe_shape_t& s) { return s.H >= 512 && s.F >= 512 ? 0 : 1; }

// Upper bound on the tiles of one kind: experts of this kind, one tile each,
// and the base kind's further tiles.
inline int64_t mx_tiles(const moe_shape_t& s, int kind)
{
    const int64_t N = (int64_t)s.T * s.k;
    const int base = mx_base(s);
    if (kind < base) return 0;
    int64_t tiles = N / (kind + 1 == kMxKinds ? 1 : mx_rows(kind + 1) + 1);
    if (tiles > s.E) tiles = s.E;
    return kind == base ? tiles + N / mx_rows(base) : tiles;
}

// Upper bound on the K-parts of one kind in one launch: no more than the
// workgroups (more parts than that, up to three rounds of them, were no faster
// on one decoded token's 96 tiles), and than its tiles cut into parts of
// kMxMinStages.
inline int64_t mx_part_units(const moe_shape_t& s, int kind)
{
    const int64_t tiles = mx_tiles(s, kind);
    const int64_t gu = tiles * (s.F / (kMxTileN / 2)) * (s.H / kMxStage / kMxMinStages);
    const int64_t dn = tiles * ((s.H + kMxTileN - 1) / kMxTileN) * (s.F / kMxStage / kMxMinStages);
    const int64_t u = gu > dn ? gu : dn;
    return u < kGemmMaxGrid ? u : kGemmMaxGrid;
}

struct MxWsLayout {
    size_t sched, vrow, h, hs, part[kMxKinds], total;
};
inline MxWsLayout mx_ws_layout(const moe_shape_t& s)
{
    const size_t N = (size_t)s.T * s.k, n1 = N > 0 ? N : 1;
    MxWsLayout w;
    size_t o = 0;
    w.sched = o; o = align256(o + (size_t)((kMxKinds + 1) * (s.E + 1)) * 4);
    w.vrow = o;  o = align256(o + n1 * 4);
    w.h = o;     o = align256(o + n1 * s.F);
    w.hs = o;    o = align256(o + n1 * (s.F / kMxBlock));
    for (int k = 0; k < kMxKinds; ++k) {
        w.part[k] = o;
        o = align256(o + (size_t)mx_part_units(s, k) * mx_rows(k) * kMxTileN * 4);
    }
    w.total = o;
    return w;
}

// Workgroups of the norm's backward, each with its own fp32 sums of dweight. The
// sums are G x H x 4 bytes written and read, beside the rows' T x H x 8 in bf16:
// 7168 columns with the second gradient, 8192 rows 86 us, 2048 25 us, 1024 17 us (5.5,
// 4.7, 3.4 TB/s of the rows).
constexpr int kNormBwdGroups = 512;
inline int norm_bwd_groups(const moe_shape_t& s)
{
    return s.T < kNormBwdGroups ? s.T : kNormBwdGroups;
}

}  // namespace moe

hipError_t moe_launch_rmsnorm(const moe_shape_t& s, const void* x, const void* residual,
                              const void* weight, float eps, void* s_out, void* y, void* q,
                              void* scales, float* rstd, hipStream_t st);
hipError_t moe_launch_rmsnorm_backward(const moe_shape_t& s, const void* s_in, const void* weight,
                                       const float* rstd, const void* dy, const void* ds, void* dx,
                                       float* dweight, float* part, hipStream_t st);
hipError_t moe_launch_mx_quantize(int64_t rows, int64_t cols, int dtype, const void* x, void* q,
                                  void* scales, hipStream_t st);
hipError_t moe_launch_permute_mx(const moe_shape_t& s, const void* q, const void* scales,
                                 const int32_t* ids, const int32_t* eidx, const int32_t* plan,
                                 void* buf_q, void* buf_s, int32_t* dest_row, int32_t* row_src,
                                 hipStream_t st);
struct MoeMxWeights {
    const uint8_t *gate, *gate_s, *up, *up_s, *down, *down_s;
};
hipError_t moe_launch_grouped_gemm_mx(const moe_shape_t& s, const void* a, const void* a_s,
                                      const int32_t* plan, const MoeMxWeights& w, void* y,
                                      char* ws, hipStream_t st);
size_t moe_grad_ws_bytes(int n, const moe_grad_t* g);
hipError_t moe_launch_grad_norm(int n, const moe_grad_t* g, float* norm, int32_t* err, double* part,
                                hipStream_t st);
hipError_t moe_launch_grad_clip(int n, const moe_grad_t* g, float max_norm, const float* norm,
                                hipStream_t st);
