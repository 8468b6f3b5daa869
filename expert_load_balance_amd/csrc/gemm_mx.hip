// gemm_mx.hip -- the grouped SwiGLU expert GEMM on 8-bit blocks (serving), with
// weights in 8-bit or 4-bit blocks (WB).
//
//   gate/up: h = blocks(silu(Wg a) * (Wu a)), 32 columns of h to a scale;
//   down:    y = Wd h, rounded to bf16.
//
// Products run on v_mfma_scale_f32_32x32x64_f8f6f4: e4m3 codes with a
// power-of-two scale per 32 values of K, applied inside the instruction, so
// no scaling is left for the vector unit. Lane l of an operand holds row
// l % 32; with K cut into 16-byte chunks, lanes 0..31 hold chunks 0 and 2 of
// the 64 and lanes 32..63 chunks 1 and 3, and the scale of 32-value block b
// comes from lanes 32 b .. 32 b + 31. Weights are the first operand, so a
// lane's 16 results are one token's columns 8 (i / 4) + 4 (l / 32) + i % 4 of
// a 32-column block. The instruction adds the products of 8 neighbouring K
// values as integers, cut toward zero at 2^-13 of the largest exponent among
// the eight, and the eights' sums in fp32: its results carry about 18 bits of
// the magnitudes added where values differ by a few binades, 11 at worst. The
// unscaled 8-bit instruction (half the rate) cuts the same way.
//
// Expert e's rows are its pieces in rank order (virtual rows). Up to 32, 64 or
// 128 of them are one tile of kind 3, 2 or 1: such a group only streams its
// weights, and small tiles keep more of the LDS for copies in flight. More are
// shared evenly by tiles of at most 256 (kind 0; 128, kind 1, where K is below
// 512 values). A persistent workgroup of four waves per CU takes tiles of rows x
// 256 weight rows in the order kind, expert, N-tile, M-tile; tile j goes to
// workgroup slot j mod P, slots numbered so that one XCD holds neighbours (they
// share rows and weights in its L2). Kinds follow each other in one numbering,
// so a workgroup's total differs from another's by about one tile whatever the
// mix.
//
// The leftover tiles of a kind past its whole rounds of P are cut along K
// when the launch has fewer than kSplitRounds rounds of tiles (on 1.5 rounds
// of the 8-expert shape's down projection 377 -> 285 us with the fixup; from 4
// rounds up it gained what the fixup cost): each part stores its fp32 tile in
// fragment order, and mx_fixup_kernel adds the parts in order and finishes.
//
// Measured (us, gate/up then down, whole launches without the fixups, in a stream
// of calls once the clock has settled):
//   8 rows of 8 experts, 4096 x 1536      26 and 14     (3.9 TB/s of weights)
//   2048 rows of 128 experts, 4096 x 1536 273 and 149   (6.1 and 5.6 TB/s)
//   32768 rows of 128 experts, 2048 x 768 160 and 103   (1.29 and 1.00 PFLOP/s)
//   4094 rows of 8 experts, 4096 x 14336  474 and 250   (2.03 and 1.92 PFLOP/s)
//   65536 rows of 256 experts, 7168 x 2048 2211 and 1214 (1.74 and 1.58 PFLOP/s)
// The first two are bound by streaming the weights. The last two are bound by
// copies and products that overlap in part only, at a clock that the chip's power
// holds down (see the 256-row tiles below). In the middle one six to sixteen
// stages a tile hide neither its cold start nor its epilogue, which takes 5 to 7 us a
// tile: the vector unit's silu and quantisation of 128 values a lane in gate/up
// (whose 32 KB of a tile are no load on the memory), y's writes in down.
//
// 4-bit weights (half the bytes; the instruction takes as long, an 8-bit operand sets
// its rate):
//   2048 rows of 128 experts, 4096 x 1536 176 and 87    (4.9 TB/s of weights)
//   4094 rows of 8 experts, 4096 x 14336  412 and 220   (2.33 and 2.19 PFLOP/s)
//   65536 rows of 256 experts, 7168 x 2048 1860 and 1115 (2.07 and 1.73 PFLOP/s)
// The first is bound by what a stage of a small tile does in turn (copies out, reads,
// splitting the rows' codes, products) on one wave a SIMD.
//
// Registers: the 256-row kernels fill the vector registers (244 in gate/up and 252 in
// down, and 256 accumulators; 216 on 4-bit weights) and spill scalars to lanes of vector
// registers, held across a tile's stages for the code between tiles. On 8-bit weights
// these are 128 (gate/up) and 115 (down), the stages' own addresses not among them; on
// 4-bit weights 362 and 195, of which a stage of the small tiles reads up to 19 back (gate/up
// of 32 rows). The 8-bit down kernels keep 20 bytes a lane in scratch, the 4-bit one without
// 256-row tiles 36.
#include <type_traits>
#include <utility>

#include "lds_pipe.h"
#include "step.h"

namespace {

using namespace moe::lds;
using moe::kMxKinds;
using moe::mx_rows;

constexpr int kThreads = 256;
constexpr int kTN = moe::kMxTileN;
constexpr int kTK = moe::kMxStage;
constexpr int kSplitRounds = 3;
constexpr int kNothing = 0x7fffffff;     // stages of the stream past the last unit
constexpr int kPieces = 4;               // of an expert, loaded ahead of their number
enum { kGateUp = 0, kDown = 1 };

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// schedule (int32): for each kind the prefix of the experts' tiles [E + 1],
// then the prefix of their rows [E + 1]. Every workgroup computes it, the
// first writes it, and workgroup b fills vrow[256 b ..], the buffer row of
// each virtual row.
__global__ __launch_bounds__(kThreads) void mx_schedule_kernel(int E, int R, int N, int base,
                                                               const int32_t* __restrict__ plan,
                                                               int32_t* __restrict__ sched,
                                                               int32_t* __restrict__ vrow)
{
    __shared__ int32_t sum[kMxKinds + 1][kThreads / 64];
    __shared__ int32_t rs[kThreads + 1];
    const moe::PlanLayout L = moe::plan_layout(E, R);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int c = 0;
    if (tid < E) {
        // (the first pieces are loaded beside their number, which says how many count)
        int n[kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) n[p] = p < R ? plan[L.piece_cnt + (size_t)tid * R + p] : 0;
        const int np = plan[L.piece_num + tid];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) c += p < np ? n[p] : 0;
        for (int p = kPieces; p < np && p < R; ++p) c += plan[L.piece_cnt + (size_t)tid * R + p];
    }
    // an expert's rows are of one kind: whole tiles and a tail of kind `base`,
    // or, where they fit a smaller tile, one of that kind
    int v[kMxKinds + 1];
#pragma unroll
    for (int k = 0; k < kMxKinds; ++k) {
        const int below = k + 1 < kMxKinds ? mx_rows(k + 1) : 0;
        const bool mine = k < base ? false : k == base ? c > below : c > below && c <= mx_rows(k);
        v[k] = mine ? (c + mx_rows(k) - 1) / mx_rows(k) : 0;
    }
    v[kMxKinds] = c;
    // inclusive prefixes: within the waves, then the waves before
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
#pragma unroll
        for (int q = 0; q <= kMxKinds; ++q) {
            const int up = __shfl_up(v[q], off);
            v[q] += lane >= off ? up : 0;
        }
    if (lane == 63)
#pragma unroll
        for (int q = 0; q <= kMxKinds; ++q) sum[q][wave] = v[q];
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64 - 1; ++w)
#pragma unroll
        for (int q = 0; q <= kMxKinds; ++q) v[q] += w < wave ? sum[q][w] : 0;
    if (blockIdx.x == 0)
#pragma unroll
        for (int q = 0; q <= kMxKinds; ++q) {
            if (tid == 0) sched[q * (E + 1)] = 0;
            if (tid < E) sched[q * (E + 1) + tid + 1] = v[q];
        }
    if (tid == 0) rs[0] = 0;
    rs[tid + 1] = v[kMxKinds];
    __syncthreads();
    const int x = blockIdx.x * kThreads + tid;
    if (x >= N) return;
    int lo = 0, hi = E - 1;  // the expert whose rows hold x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (rs[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    const int at = x - rs[lo];
    int n[kPieces], r0[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        n[p] = p < R ? plan[L.piece_cnt + (size_t)lo * R + p] : 0;
        r0[p] = p < R ? plan[L.piece_row + (size_t)lo * R + p] : 0;
    }
    const int np = plan[L.piece_num + lo];
    int cum = 0, row = -1;
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
        if (p < np) {
            if (row < 0 && at < cum + n[p]) row = r0[p] + (at - cum);
            cum += n[p];
        }
    for (int p = kPieces; p < np && p < R && row < 0; ++p) {
        const int m = plan[L.piece_cnt + (size_t)lo * R + p];
        if (at < cum + m) row = plan[L.piece_row + (size_t)lo * R + p] + (at - cum);
        cum += m;
    }
    // (rows past the plan's total, or a damaged plan, stay in the buffer)
    vrow[x] = row >= 0 && row < N ? row : 0;
}

// silu(z) = z / (1 + e^-z) with the hardware exp2 and reciprocal (about 1 ulp
// each); h is rounded to 4 bits right after.
__device__ __forceinline__ float fast_silu(float z)
{
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

__device__ __forceinline__ i32x8 frag(const char* p0, const char* p1)
{
    const u32x4 a = *reinterpret_cast<const u32x4*>(p0), b = *reinterpret_cast<const u32x4*>(p1);
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// A weight operand of 64 values: 8-bit codes as a row's, 4-bit ones in half of
// the registers.
template <int WB>
__device__ __forceinline__ i32x8 wfrag(const char* p0, const char* p1)
{
    if constexpr (WB == 8) return frag(p0, p1);
    const u32x4 a = *reinterpret_cast<const u32x4*>(p0);
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
}

// acc += W T over one 64-value k-step, with the scales in byte B of ws and ts.
template <int WB, int B>
__device__ __forceinline__ f32x16 mfma(const i32x8& w, const i32x8& t, const f32x16& acc, uint32_t ws, uint32_t ts)
{
    // (operand formats: 0 is e4m3, 4 is e2m1)
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, t, acc, WB == 8 ? 0 : 4, 0, B, (int)ws, B, (int)ts);
}

// 16 codes to bf16, times their scale (the word's byte B as an exponent):
// exact for scales 2^-124 .. 2^119; below, bf16's subnormals drop bits of
// values under 2^-126.
struct Bf16x16 {
    bf16x8 lo, hi;
};
template <int B>
__device__ __forceinline__ Bf16x16 widen(const u32x4& c, uint32_t scales)
{
    const uint32_t at = B == 3 ? scales >> 1 : scales << (B == 3 ? 0 : 23 - 8 * B);
    const float s = __uint_as_float(at & 0x7f800000u);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, false));
        w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, true));
    }
    return Bf16x16{__builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]}),
                   __builtin_bit_cast(bf16x8, u32x4{w[4], w[5], w[6], w[7]})};
}

// The codes of a word whose exponent is 8 and more (of 15), the others 0. The
// byte masks are the top exponent bits, spread by the permute's sign selectors.
__device__ __forceinline__ uint32_t upper_codes(uint32_t v)
{
    return v & __builtin_amdgcn_perm(v << 9, v << 1, 0x090b080au);
}

// (a, b) -> lanes 0..31: (a, a of the lane 32 up); lanes 32..63: (b of the
// lane 32 down, b).
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b)
{
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(a, b, false, false));
    a = r[0];
    b = r[1];
}

// One accumulator, read where this stands: the accumulators fill the second
// half of the register file, and read as ordinary values they would be moved
// out of it all at once, ahead of their uses. drain() comes before the first
// read: the matrix pipe's results need up to 19 cycles (16-pass instructions)
// after the last one was issued, which the compiler counts for its own
// reads only.
__device__ __forceinline__ float take(float a)
{
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}
__device__ __forceinline__ void drain()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Stores through a buffer descriptor: a lane whose offset is kZeroRow (a
// padding row, a column past the end) stores nothing, without a branch, so
// that the epilogue is one block and the accumulators are read where they are
// needed.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t store_to(void* base)
{
    return __builtin_amdgcn_make_buffer_rsrc(uni_ptr((char*)base), 0, (int)kCopyRange, 0x00020000);
}
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, uint32_t a, uint32_t b, uint32_t c,
                                        uint32_t d)
{
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{a, b, c, d}, rsrc, (int)off, 0, 0);
}

// h of one token's 32-column block from the lane's 16 columns (the lane 32
// away holds the other 16): quantised, 16 consecutive codes stored per lane.
__device__ __forceinline__ void store_h(const f32x16& g, const f32x16& u, __amdgpu_buffer_rsrc_t h, uint32_t off,
                                        __amdgpu_buffer_rsrc_t hs, uint32_t soff, int half)
{
    float hv[16];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        hv[i] = fast_silu(take(g[i])) * take(u[i]);
        top = max(top, moe::mx_mag(hv[i]));
    }
    uint32_t t0 = top, t1 = top;
    swap32(t0, t1);
    const uint32_t byte = moe::mx_scale_byte(max(t0, t1));
    uint32_t w[4];  // w[i]: columns 8 i + 4 half ..
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = moe::mx_pack4(hv[4 * i], hv[4 * i + 1], hv[4 * i + 2], hv[4 * i + 3], byte);
    swap32(w[0], w[2]);  // lower lanes: columns 0..3, 4..7; upper: 16..19, 20..23
    swap32(w[1], w[3]);
    store16(h, off, w[0], w[2], w[1], w[3]);
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)byte, hs, (int)(half ? kZeroRow : soff), 0, 0);
}

// y of one token's 32-column block: 8 consecutive bf16 columns per store. bf16,
// since y is the combine's input, which has the layer's type: fp32 rows would
// double the down projection's writes and the combine's reads (0.94 GB each for
// 65536 rows of 7168). The combine adds in fp32 and rounds its sum again, so
// its output is 0.0024 of its norm off where one rounding is 0.0017.
__device__ __forceinline__ void store_y(const f32x16& a, __amdgpu_buffer_rsrc_t y, uint32_t off)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t e[2], o[2];  // columns 16 i + 4 half .., 16 i + 8 + 4 half ..
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            e[q] = moe::pack_bf16x2(take(a[8 * i + 2 * q]), take(a[8 * i + 2 * q + 1]));
            o[q] = moe::pack_bf16x2(take(a[8 * i + 4 + 2 * q]), take(a[8 * i + 4 + 2 * q + 1]));
            swap32(e[q], o[q]);
        }
        store16(y, off == kZeroRow ? off : off + 32 * i, e[0], e[1], o[0], o[1]);
    }
}

// The same value through an opaque move: what is computed from it stays
// where it is written, instead of being hoisted out of the unit loop to hold
// registers across it.
__device__ __forceinline__ int opaque_v(int v)
{
    int r;
    asm volatile("v_mov_b32 %0, %1" : "=v"(r) : "v"(v));
    return r;
}

// A constant in a scalar register of its own: where a value per lane needs the
// same constant, the compiler would take both from one vector register, and
// all that follows from the scalar one with it.
template <int V>
__device__ __forceinline__ int scalar()
{
    int r;
    asm volatile("s_mov_b32 %0, %1" : "=s"(r) : "i"(V));
    return r;
}

// ------------------------------------------------------------ work units --

// Units of one kind: `full` whole tiles, then L leftover tiles in S K-parts
// of at least kMxMinStages stages (S == 1: whole), or in two parts of their rows
// (halves). first: their place in the launch's numbering.
struct KindWork {
    int full, L, S, first, count, halves;
};
// rest: the tiles of the kinds behind this one (kind 0 only).
__device__ __forceinline__ KindWork kind_work(int n, int first, int P, int KT, bool split, bool whole, int rest)
{
    KindWork w{n, 0, 1, first, n, 0};
    const int left = uni(n % P);
    if (left > 0 && split) {
        const int s0 = uni(min(P / left, KT / moe::kMxMinStages));
        if (s0 > 1) {
            w.S = s0;
            w.L = left;
            w.full = n - left;
            w.count = w.full + w.L * w.S;
        }
    }
    // A last round less than half full: its 256-row tiles take half of their
    // rows on the workgroups that would have none (4.4 rounds of the 128-expert
    // layer's 4096 tokens: 335 -> 324 us for the whole call; from 8 rounds up no
    // difference).
    if (!whole && w.S == 1 && left > 0 && 2 * left + rest <= P) {
        w.halves = 1;
        w.L = left;
        w.full = n - left;
        w.count = w.full + 2 * left;
    }
    return w;
}

struct Unit {
    int e, n0, rows, x0;   // expert, first weight row, rows, first virtual row
    int k0, KT, pidx;      // K-stages k0 .. k0 + KT; partial tile or -1
    int rot;               // which of them comes first (the others follow, then 0 .. rot - 1)
    int alone;             // the expert has no other M-tile
};

// Stages that K values take: of 128 values, and in the small tiles of 4-bit
// weights of 256, so that a stage takes whole 128-byte lines of every weight row
// (the last one may be half). With 64 bytes of a row a stage and the copies
// streamed, a line was fetched again for its other half: 256 tokens of 128 experts of
// 4096 x 1536, gate/up 251 us, down 139.
template <int KIND, int WB>
__device__ __forceinline__ int stages(int K)
{
    return WB == 4 && KIND > 0 ? (K + 2 * kTK - 1) / (2 * kTK) : K / kTK;
}

struct Gemm {
    int E, ntn, H, F, P, N;
    int split;                  // tiles may be cut along K
    const uint8_t *a, *as;
    const int32_t *sched, *vrow;
    const uint8_t *w0, *s0, *w1, *s1;
    uint8_t *h, *hs;
    uint16_t* y;
    float* part[kMxKinds];
};

// The launch's arguments (the kernel's first argument is a Gemm), read again
// where this stands: they serve between tiles only, and held across a tile's
// stages they would push the addresses that the stages need out of the scalar
// registers.
__device__ __forceinline__ Gemm again()
{
#ifdef __HIP_DEVICE_COMPILE__
    typedef const __attribute__((address_space(4))) Gemm constant;
    constant* p = (constant*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *p;
#else
    return Gemm{};
#endif
}

// The units of kinds 0 .. KIND - 1 come first.
template <int MODE, int WB>
__device__ __forceinline__ KindWork work_of(const Gemm& g, int kind)
{
    const int K = MODE == kGateUp ? g.H : g.F;
    KindWork w{0, 0, 1, 0, 0, 0};
    int n[kMxKinds], total = 0, first = 0;
#pragma unroll
    for (int k = 0; k < kMxKinds; ++k) total += n[k] = ldc(g.sched, k * (g.E + 1) + g.E) * g.ntn;
#pragma unroll
    for (int k = 0; k < kMxKinds; ++k)
        if (k <= kind) {
            w = kind_work(n[k], first, g.P, k == 0 ? stages<0, WB>(K) : stages<1, WB>(K), g.split && total < kSplitRounds * g.P, k > 0, total - n[0]);
            first += w.count;
        }
    return w;
}

// Tile t of the kind in expert e, whose tiles are t0 .. t1 and rows r0 .. r1:
// N-tile, then M-tile (M fastest, so that an expert's tiles meet its weights in
// the L2 together).
template <int MODE, int KIND>
__device__ __forceinline__ void place(const Gemm& g, int t, int e, int t0, int t1, int r0, int r1, Unit& u)
{
    const int mts = t1 - t0, local = t - t0 * g.ntn, c = r1 - r0;
    // 256-row tiles share the expert's rows evenly, in whole token blocks of the
    // 2 x 2 waves: whole tiles are bound by the products and short ones by their
    // copies' latency (32 rows take 60 % of 256 rows' time), so three tiles of
    // 181 are faster than 256 + 256 + 32. Eight experts of 544 rows of 4096 x 14336:
    // gate/up 680 -> 584 us, down 309 -> 272 us.
    const int height = KIND == 0 ? (c + 64 * mts - 1) / (64 * mts) * 64 : mx_rows(KIND);
    const int nt = local / mts, v0 = local % mts * height;
    u.e = uni(e);
    u.n0 = uni(nt * (MODE == kGateUp ? kTN / 2 : kTN));
    u.rows = uni(min(height, c - v0));
    u.x0 = uni(r0 + v0);
    u.alone = uni(mts == 1);
}

// The tile's expert by the prefix of tiles: scalar loads, which do not wait
// for the copies in flight.
template <int MODE, int KIND>
__device__ __forceinline__ void tile_of(const Gemm& g, int t, Unit& u)
{
    const int32_t* ts = g.sched + KIND * (g.E + 1);
    const int32_t* rs = g.sched + kMxKinds * (g.E + 1);
    int lo = 0, hi = g.E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ldc(ts, mid) * g.ntn <= t) lo = mid;
        else hi = mid - 1;
    }
    place<MODE, KIND>(g, t, lo, ldc(ts, lo), ldc(ts, lo + 1), ldc(rs, lo), ldc(rs, lo + 1), u);
}

// The same by one round of loads over the wave, where nothing else is in
// flight yet (a launch's first units, the fixup): the search's dependent loads,
// cold after the schedule kernel, were about 4 us of every launch.
template <int MODE, int KIND>
__device__ __forceinline__ void tile_by_wave(const Gemm& g, int t, Unit& u)
{
    const int32_t* ts = g.sched + KIND * (g.E + 1);
    const int32_t* rs = g.sched + kMxKinds * (g.E + 1);
    const int lane = threadIdx.x & 63;
    int a[4], b[4], c[4], d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = min(64 * i + lane, g.E - 1);
        a[i] = ts[e];
        b[i] = ts[e + 1];
        c[i] = rs[e];
        d[i] = rs[e + 1];
    }
    int chunk = 0, at = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const uint64_t hit = __ballot(a[i] * g.ntn <= t && t < b[i] * g.ntn);
        if (hit) {
            chunk = i;
            at = __builtin_ctzll(hit);
        }
    }
    auto of = [&](const int* v) {
        return __builtin_amdgcn_readlane(chunk == 0 ? v[0] : chunk == 1 ? v[1] : chunk == 2 ? v[2] : v[3], at);
    };
    place<MODE, KIND>(g, t, 64 * chunk + at, of(a), of(b), of(c), of(d), u);
}

template <int MODE, int KIND, int WB, bool WAVE = false>
__device__ __forceinline__ Unit unit_of(const Gemm& g, const KindWork& w, int j)
{
    Unit u;
    int t = j - w.first;
    u.k0 = 0;
    u.KT = stages<KIND, WB>(MODE == kGateUp ? g.H : g.F);
    u.pidx = -1;
    int half = -1;
    if (KIND == 0 && w.halves && t >= w.full) {
        half = uni((t - w.full) / w.L);
        t = w.full + uni((t - w.full) % w.L);
    } else if (t >= w.full) {  // parts of the leftover tiles, part-major
        u.pidx = uni(t - w.full);
        const int p = uni(u.pidx / w.L), KT = u.KT;
        u.k0 = uni(p * KT / w.S);
        u.KT = uni((p + 1) * KT / w.S) - u.k0;
        t = w.full + uni(u.pidx % w.L);
    }
    if (WAVE) tile_by_wave<MODE, KIND>(g, t, u);
    else tile_of<MODE, KIND>(g, t, u);
    if (KIND == 0 && half >= 0) {
        const int h = (u.rows + 127) / 128 * 64, r0 = uni(half * h);
        u.x0 += r0;
        u.rows = uni(half == 0 ? min(h, u.rows) : max(u.rows - h, 0));
    }
    // If every workgroup walked K from the same stage, the lines in flight would
    // share their low address bits where rows are a multiple of 4 KB apart, and
    // crowd a few memory channels. So the XCDs start four stages apart (of 128
    // values a whole group of scales, and only where K has no group cut short; of
    // 256 values two groups, and the last stage may be half a one: see cut); within
    // one, tiles stay in step for what they share in its L2.
    // Measured, no stagger / by N-tile / by XCD: gate/up of 128 x 16 rows of
    // 4096 x 1536 388 / 339 / 326 us; down of 256 x 256 rows of 7168 x 2048
    // 1209 / (by N-tile on 4 KB rows only) / 1158 us; 8 x 512 rows of 4096 x 14336
    // alike within the noise.
    u.rot = u.pidx < 0 && u.KT % 4 == 0 ? uni((int)blockIdx.x % 8 * 4 % u.KT) : 0;
    return u;
}

// Waves of a workgroup tile: kind 0, 2 x 2, each 128 rows x 128 weight rows;
// smaller kinds, 1 x 4, each all rows x 64 weight rows. WB 32-row weight
// blocks per wave (gate/up: the first half of them gate, the rest the same
// columns of up) and TB 32-row token blocks.
template <int MODE, int KIND, int WB>
struct Geo {
    static constexpr int kRows = mx_rows(KIND);
    static constexpr int WM = KIND == 0 ? 2 : 1, WN = 4 / WM;
    static constexpr int TB = kRows / 32 / WM, WBL = 8 / WN;
    static constexpr int kPanels = WB == 4 && KIND > 0 ? 2 : 1;  // of 128 values of K in a stage, rows by panel
    static constexpr int kA = kRows * kTK * kPanels;
    static constexpr int kACopies = kRows / 32 * kPanels;    // 16-byte copies per wave per stage
    static constexpr int kWRow = kTK * kPanels * WB / 8;     // bytes of a weight row's stage
    static constexpr int kWBytes = kTN * kWRow;              // 32 or 16 KB of weights per stage
    static constexpr int kWCopies = kWBytes / 4096, kWBlock = kTN / kWCopies;  // copies, weight rows of one
    static constexpr int kPerStage = kWCopies + kACopies + 2;
    // LDS, kinds 1..3: slots of rows + weights, then their scales, then three
    // row lists. Kind 0: two slots of rows, a ring of 5 weight units of 128
    // rows (a stage takes two), the scales of up to four stages (16 bytes for
    // each weight row, then for each row), the lists.
    // (The scales of a stage of 256 values come as 16 bytes a row, with those of
    // its neighbour, in every other stage: 128 x 16 rows of 4096 x 1536, gate/up 189
    // -> 183 us, down 91 -> 88.)
    static constexpr int kSlot = KIND == 0 ? kA : kA + kWBytes;
    static constexpr int kScaleRow = KIND == 0 || kPanels == 2 ? 16 : 4;
    static constexpr int kScale = (kTN + kRows) * kScaleRow;
    static constexpr int kSlots = KIND == 0 ? 2 : (160 * 1024 - 3 * kRows * 4) / (kSlot + kScale) > 4
                                                      ? 4 : (160 * 1024 - 3 * kRows * 4) / (kSlot + kScale);
    static constexpr int kAhead = KIND == 0 ? 2 : kSlots - 1;  // stages copied ahead of the products
    static constexpr int kUnits = KIND == 0 ? 5 : 0, kUnit0 = kSlots * kSlot, kUnit = 128 * kWRow;
    static constexpr int kScale0 = kUnit0 + kUnits * kUnit;
    static constexpr int kList0 = kScale0 + (KIND == 0 ? 1 : kSlots) * kScale;
    static constexpr int kKept0 = kList0 + 3 * kRows * 4;      // kind 0: three units for each wave
    static constexpr int kBytes = kKept0 + (KIND == 0 ? 4 * 3 * 32 : 0);
    // Stages of a unit in the stream: at least kAhead, so that the copies are
    // never more than one unit ahead.
    __device__ static int stream_stages(int KT) { return KT < kAhead ? kAhead : KT; }
    // weight-tile row of block j's first row, for wave column wn
    __device__ static int wrow(int wn, int j)
    {
        return MODE == kGateUp ? (j / (WBL / 2)) * 128 + wn * (128 / WN) + (j % (WBL / 2)) * 32
                               : wn * (kTN / WN) + j * 32;
    }
};
constexpr int max4(int a, int b, int c, int d)
{
    const int x = a > b ? a : b, y = c > d ? c : d;
    return x > y ? x : y;
}
template <int WB>
constexpr int kLds = max4(Geo<kGateUp, 0, WB>::kBytes, Geo<kGateUp, 1, WB>::kBytes, Geo<kGateUp, 2, WB>::kBytes,
                          Geo<kGateUp, 3, WB>::kBytes);
static_assert(kLds<8> <= 160 * 1024 && kLds<4> <= 160 * 1024, "LDS");

// Place of chunk c (0..3) in a weight row of 64 bytes (4-bit codes, 256-row
// tiles): four rows fill the 256 bytes that 16 lanes read at once, so the chunks
// turn with every fourth row.
__device__ __forceinline__ int swz4(int r) { return (r >> 2) & 3; }

// Weights that one tile reads are streamed past the caches, those that the
// expert's other M-tiles read too are kept. Tiles below the launch's whole ones
// (mx_base) are their expert's only tile: gate/up of 128 x 16 rows of 4096 x 1536
// 279 -> 261 us streamed, of 256 x 32 rows of 7168 x 2048 1404 -> 1320 us. 256-row
// tiles are kept (streamed, the 256-expert layer's gate/up took 2437 us for 2331).
// Whole tiles of 128 rows (H or F below 512) are either, so there each expert goes
// by its own tiles (both projections, beside all kept / all streamed): 16 tiles of
// each of 8 experts of 4096 x 384 156 us (154 / 177), two of each of 256 experts of
// 7168 x 384 1187 us (1164 / 1221), two of each of 64 of 256 x 8192 348 us (347 / 340),
// one of each of 128 of 4096 x 384 170 us (195 / 169).
enum Weights { kKept, kStreamed, kByExpert };

// Copies of a unit's stages. The stages of a workgroup's units of one kind
// form one stream: stage number n of the stream sits in slot n % kSlots, and
// the copies run kAhead stages ahead of the products, across units. Past the
// last unit, and past the stages of a unit with fewer than kAhead, the stream
// goes on with copies of nothing, so that every stage issues the same number
// of instructions and the waits count the same.
//
// 16-byte copies (see lds_pipe.h): instruction q = wave + 4 i fills rows 8 q
// .. 8 q + 7 of an operand, lane l row 8 q + l / 8, chunk l % 8 (of weight rows
// of 64 bytes rows 16 q .. 16 q + 15, lane l row 16 q + l / 4, chunk l % 4). Scales: 4
// bytes (a stage's four blocks) of weight row 64 wave + lane and, in the
// lanes below kRows / 4, of row kRows / 4 * wave + lane.
template <int MODE, int KIND, Weights WEIGHTS, int WB>
struct Copier {
    using GE = Geo<MODE, KIND, WB>;
    static constexpr int kHalf = GE::kWCopies / 2;  // weight copies of 128 rows
    const char *ab, *wb0, *wb1, *asb, *sb;  // rows, the first and the other 128 weight rows, scales
    int upper;                              // down: weight rows from row 128 on (0 or less: none)
    uint32_t aoff[GE::kACopies], woff, asoff, wsoff;
    int block;         // bytes from a copy's weight rows to the next one's
    int rot, alone;
    int st, KT, real;  // the next stage to copy, the unit's stages in the stream, those with data
    int k0, half;      // 4-bit small tiles: the unit's first stage, its stage of 128 values only (or -1)
    uint32_t whalf;    // and woff without that stage's second half
    uint32_t arange, wrange;  // bytes of the rows' and of the expert's scales

    // list: the unit's row list in LDS (gate/up; down reads h in virtual order)
    __device__ __forceinline__ void setup(const Gemm& g, const Unit& u, const int32_t* list, int wave, int lane)
    {
        const int K = MODE == kGateUp ? g.H : g.F, KS = K / moe::kMxBlock, wrows = MODE == kGateUp ? g.F : g.H;
        const size_t e0 = (size_t)u.e * wrows;
        const size_t x0 = MODE == kGateUp ? 0 : (size_t)u.x0;
        // (in the down projection's last tile the other 128 rows may lie past
        // the matrix)
        upper = wrows - u.n0 - kTN / 2;
        ab = uni_ptr((const char*)g.a + x0 * K + u.k0 * (kTK * GE::kPanels));
        const int KB = K * WB / 8;  // bytes of a weight row
        wb0 = uni_ptr((const char*)g.w0 + e0 * KB + u.k0 * GE::kWRow);
        wb1 = uni_ptr((const char*)(MODE == kGateUp ? g.w1 : g.w0) + e0 * KB + u.k0 * GE::kWRow);
        const int s0 = GE::kPanels == 1 ? u.k0 * 4 : 0;
        asb = uni_ptr((const char*)g.as + x0 * KS + s0);
        sb = uni_ptr((const char*)(MODE == kGateUp && wave >= 2 ? g.s1 : g.s0) + e0 * KS + s0);
        if constexpr (GE::kPanels == 2) {
            k0 = u.k0;
            half = K % (2 * kTK) ? stages<KIND, WB>(K) - 1 - u.k0 : -1;
            // (a group of 16 bytes may reach past a row's end, and the last row's past the
            // array; of h no more than a tile's rows and the next one, so that the range stays
            // within 32 bits, whatever N * KS is: N * H is below 2^31, N * F below 2^40)
            const int rows = MODE == kGateUp ? g.N : min(g.N - (int)x0, GE::kRows + 1);
            arange = uni((int)((uint32_t)rows * (uint32_t)KS));
            wrange = uni((int)((uint32_t)wrows * (uint32_t)KS));
        }
        st = scalar<0>();
        rot = u.rot;
        if (WEIGHTS == kByExpert) alone = u.alone;
        real = u.KT;
        KT = GE::stream_stages(u.KT);
        // (looked up for padding rows too: as a load under a condition it would be
        // a branch, and what is set beside it a value per lane)
        auto source = [&](int r) {
            uint32_t x = MODE == kGateUp ? (uint32_t)list[r] : (uint32_t)r;
            asm volatile("" : "+v"(x));
            return x;
        };
        auto weight = [&](int r) {
            return (uint32_t)(MODE == kGateUp ? u.n0 + (r & 127) : min(u.n0 + r, wrows - 1));
        };
#pragma unroll
        for (int i = 0; i < GE::kACopies; ++i) {
            const int r = 8 * (wave + 4 * (i % (GE::kRows / 32))) + (lane >> 3);
            const uint32_t off = source(r) * (uint32_t)K + (uint32_t)(((lane & 7) ^ swz(r)) * 16);
            aoff[i] = r < u.rows ? off : kZeroRow;
        }
        const int r0 = GE::kWRow == 128 ? 8 * wave + (lane >> 3) : 16 * wave + (lane >> 2);
        const int chunk = GE::kWRow == 128 ? (lane & 7) ^ swz(r0) : (lane & 3) ^ swz4(r0);
        woff = (uint32_t)(u.n0 + r0) * (uint32_t)KB + (uint32_t)(chunk * 16);
        if constexpr (GE::kPanels == 2) whalf = chunk < 4 ? woff : kZeroRow;
        block = GE::kWBlock * KB;
        const int ar = GE::kRows / 4 * wave + lane % (GE::kRows / 4);
        const uint32_t aso = source(ar) * (uint32_t)KS;
        asoff = lane < GE::kRows / 4 && ar < u.rows ? aso : kZeroRow;
        wsoff = weight(64 * wave + lane) * (uint32_t)KS;
    }
    __device__ __forceinline__ void nothing()
    {
        st = real = rot = scalar<0>();
        KT = kNothing;
    }
    __device__ __forceinline__ int ks() const { return st + rot >= real ? st + rot - real : st + rot; }
    // A stage past the unit's last is a copy of nothing (a unit of kind 0 has at
    // least four stages, so only the last unit has such). As a comparison of a
    // scalar where it is used: a range that came round the loop would be kept
    // in a vector register.
    __device__ __forceinline__ uint32_t range() const { return (KIND == 0 ? KT != kNothing : st < real) ? kCopyRange : 0u; }
    // Of 4-bit weights the compiler keeps the stage in a vector register.
    __device__ __forceinline__ static int held(int v) { return WB == 8 ? v : uni(v); }
    // The next stage into a slot; each call of row and weight is one
    // instruction, scales is two or none.
    __device__ __forceinline__ void row(int i, uint32_t slot, int wave) const
    {
        if constexpr (GE::kPanels == 1) {
            copy16(buffer_of(ab, range()), aoff[i], held(ks() * kTK), slot + wave * 1024 + i * 4096);
        } else {
            const int panel = i / (GE::kRows / 32);
            copy16(buffer_of(ab, panel && ks() == half ? 0u : range()), aoff[i], held((2 * ks() + panel) * kTK),
                   slot + wave * 1024 + i * 4096);
        }
    }
    template <bool STREAM>
    __device__ __forceinline__ void weight(int i, uint32_t unit, int wave) const  // unit: kWBlock rows, 4 KB
    {
        const int at = ks() * GE::kWRow + (MODE == kGateUp ? i % kHalf : i) * block;
        uint32_t off = woff;
        if constexpr (GE::kPanels == 2) off = ks() == half ? whalf : woff;
        copy16<STREAM>(buffer_of(i < kHalf ? wb0 : wb1, i < kHalf || MODE == kGateUp || upper > 0 ? range() : 0u), off,
               held(at), unit + wave * 1024);
    }
    // Whether the next stage's copies have scales: of stages of 256 values the even
    // ones and a unit's first (a unit that starts elsewhere than at 0 keeps their
    // order, so an odd stage follows the even one whose copy holds its scales).
    __device__ __forceinline__ bool scaled() const
    {
        return GE::kPanels == 1 || (st < real && (st == 0 || ((k0 + ks()) & 1) == 0));
    }
    __device__ __forceinline__ void scales(uint32_t sslot, int wave, int lane) const
    {
        if constexpr (GE::kPanels == 1) {
            copy4(buffer_of(sb, range()), wsoff, ks() * 4, sslot + wave * 256);
            if (lane < GE::kRows / 4) copy4(buffer_of(asb, range()), asoff, ks() * 4, sslot + kTN * 4 + wave * GE::kRows);
        } else {  // 512 values' worth, of which the stage's are the first or the second half
            const int at = held((k0 + ks()) / 2 * 16);
            if (!scaled()) return;
            copy16(buffer_of(sb, wrange), wsoff, at, sslot + wave * 1024);
            if (lane < GE::kRows / 4) copy16(buffer_of(asb, arange), asoff, at, sslot + kTN * 16 + wave * GE::kRows * 4);
        }
    }
    // The same in pieces, in the same order: weights, rows, scales.
    template <int I>
    __device__ __forceinline__ void piece(uint32_t slot, uint32_t sslot, int wave, int lane)
    {
        if constexpr (I < GE::kWCopies) {
            if (WEIGHTS == kStreamed || (WEIGHTS == kByExpert && alone)) weight<true>(I, slot + GE::kA + I * 4096, wave);
            else weight<false>(I, slot + GE::kA + I * 4096, wave);
        } else if constexpr (I < GE::kWCopies + GE::kACopies) {
            row(I - GE::kWCopies, slot, wave);
        } else {
            scales(sslot, wave, lane);
            ++st;
        }
    }
    __device__ __forceinline__ void stage(uint32_t slot, uint32_t sslot, int wave, int lane)
    {
        if (WEIGHTS == kStreamed || (WEIGHTS == kByExpert && alone)) {
#pragma unroll
            for (int i = 0; i < GE::kWCopies; ++i) weight<true>(i, slot + GE::kA + i * 4096, wave);
        } else {
#pragma unroll
            for (int i = 0; i < GE::kWCopies; ++i) weight<false>(i, slot + GE::kA + i * 4096, wave);
        }
#pragma unroll
        for (int i = 0; i < GE::kACopies; ++i) row(i, slot, wave);
        scales(sslot, wave, lane);
        ++st;
    }
};

// The unit's row list (virtual -> buffer rows) to LDS: one copy instruction
// per wave.
template <int KIND>
__device__ __forceinline__ void copy_list(const Gemm& g, const Unit& u, uint32_t lds, int wave, int lane)
{
    constexpr int kRows = mx_rows(KIND);
    const int r = kRows / 4 * wave + lane;
    if (lane < kRows / 4)
        copy4(buffer_of(g.vrow + u.x0, kCopyRange), r < u.rows ? (uint32_t)r * 4u : kZeroRow, 0, lds + kRows * wave);
}

// A finished tile: acc[j] of token block i, weight block j.
template <int MODE, int KIND>
__device__ __forceinline__ void finish(const Gemm& g, const Unit& u, int i,
                                       const f32x16 (&acc)[Geo<MODE, KIND, 8>::WBL], const int32_t* list,
                                       int wave, int lane)
{
    using GE = Geo<MODE, KIND, 8>;  // (its waves' blocks are the same for every weight)
    const int fr = lane & 31, half = lane >> 5, wm = wave / GE::WN, wn = wave % GE::WN;
    const int r = (i * GE::WM + wm) * 32 + fr;
    const bool in = r < u.rows;
    if (MODE == kGateUp) {
        const int SF = g.F / moe::kMxBlock;
        const auto h = store_to(g.h + (size_t)u.x0 * g.F);
        const auto hs = store_to(g.hs + (size_t)u.x0 * SF);
#pragma unroll
        for (int j = 0; j < GE::WBL / 2; ++j) {
            const int col = u.n0 + GE::wrow(wn, j);
            store_h(acc[j], acc[j + GE::WBL / 2], h, in ? (uint32_t)(r * g.F + col + 16 * half) : kZeroRow, hs,
                    in ? (uint32_t)(r * SF + col / moe::kMxBlock) : kZeroRow, half);
        }
    } else {
        // (H is a multiple of 128, so a 32-column block is in or out)
        const auto y = store_to(g.y);
        const uint32_t row = (uint32_t)list[in ? r : 0] * (uint32_t)g.H * 2u + 16u * half;
#pragma unroll
        for (int j = 0; j < GE::WBL; ++j) {
            const int col = u.n0 + GE::wrow(wn, j);
            store_y(acc[j], y, in && col < g.H ? row + 2u * col : kZeroRow);
        }
    }
}

// A K-part's fp32 tile in fragment order: whole 1 KB stores, and the fixup
// finds each lane's values where the products left them.
template <int MODE, int KIND>
__device__ __forceinline__ float4* part_at(const Gemm& g, int pidx, int wave, int i, int j, int lane)
{
    using GE = Geo<MODE, KIND, 8>;
    float* base = g.part[KIND] + (size_t)pidx * GE::kRows * kTN;
    return reinterpret_cast<float4*>(base) + ((((size_t)wave * GE::TB + i) * GE::WBL + j) * 4) * 64 + lane;
}
template <int MODE, int KIND>
__device__ __forceinline__ void store_part(const Gemm& g, const Unit& u, int i,
                                           const f32x16 (&acc)[Geo<MODE, KIND, 8>::WBL], int wave, int lane)
{
    using GE = Geo<MODE, KIND, 8>;
    const bool in = (i * GE::WM + wave / GE::WN) * 32 + (lane & 31) < u.rows;  // padding rows are left out
    const auto to = store_to(part_at<MODE, KIND>(g, u.pidx, wave, i, 0, 0));
#pragma unroll
    for (int j = 0; j < GE::WBL; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            store16(to, in ? (uint32_t)(((j * 4 + q) * 64 + lane) * 16) : kZeroRow, __float_as_uint(take(acc[j][4 * q])),
                    __float_as_uint(take(acc[j][4 * q + 1])), __float_as_uint(take(acc[j][4 * q + 2])),
                    __float_as_uint(take(acc[j][4 * q + 3])));
}

// ------------------------------------------------- tiles below 256 rows --
// Bound by streaming the weights: a ring of up to four stages, one barrier per
// stage, the fragments read as the products need them. 128 experts of 16 rows
// of 4096 x 1536: 6.1 TB/s of weights, where a plain read of 4 GB reaches 6.2.
template <int I>
using Number = std::integral_constant<int, I>;
// f(0), f(1), ... with the number as a constant.
template <typename F, int... J>
__device__ __forceinline__ void unrolled(F f, std::integer_sequence<int, J...>)
{
    (f(Number<J>{}), ...);
}

template <int MODE, int KIND, Weights WEIGHTS, int WB>
__device__ __forceinline__ void ring_tiles(const Gemm& g, char* lds, int slot_id)
{
    using GE = Geo<MODE, KIND, WB>;
    // Gate and up of up to 64 rows are multiplied in bf16, which is exact: the
    // 8-bit instruction's cut leaves g and u about 1e-4 off, which sends 0.2 %
    // of h's codes to the other side of their rounding (y is then 0.0024 of its norm
    // off, with exact g and u 0.0017, which is bf16's rounding alone). Beside the
    // weights' streaming the slower products cost nothing at these sizes. On 128 rows they
    // would: 256 x 128 rows of 7168 x 2048 1585 -> 2423 us. The down projection's
    // cut reaches y without a rounding in between, and exact products there
    // would take 1 % on 32-row tiles and 10 % on 64 (256 x 64 rows: 748 -> 827 us).
    // With 4-bit weights the rows' codes are multiplied in two parts instead, those
    // of exponent 8 and more and the others: the products of a part differ by 10
    // binades at most, of which the cut takes 9. The time for a stage is half, and
    // the widening's conversions would show: 128 x 16 rows of 4096 x 1536, gate/up
    // 160 us in one part, 181 in two, 203 in bf16.
    constexpr bool kWide = WB == 8 && MODE == kGateUp && KIND >= 2, kSplit = WB == 4 && MODE == kGateUp && KIND >= 2;
    const KindWork work = work_of<MODE, WB>(g, KIND);
    const int end = work.first + work.count, P = g.P;
    // this workgroup's first unit of the kind
    int j = work.first + uni((slot_id - work.first % g.P + g.P) % g.P);
    if (j >= end) return;

    const int tid = threadIdx.x, wave = uni(tid >> 6), lane = tid & 63;
    const int fr = lane & 31, half = lane >> 5, wn = wave;
    const uint32_t lds_u = (uint32_t)(uintptr_t)lds;
    auto list = [&](int m) { return reinterpret_cast<const int32_t*>(lds + GE::kList0 + m % 3 * GE::kRows * 4); };
    auto list_u = [&](int m) { return lds_u + GE::kList0 + m % 3 * GE::kRows * 4; };

    // what the previous kind left in flight has landed, in every wave
    wait_vm_lgkm<0>();
    slot_barrier();
    Unit u = unit_of<MODE, KIND, WB, true>(g, work, j), un = u;
    copy_list<KIND>(g, u, list_u(0), wave, lane);
    bool more = j + g.P < end;
    if (more) {
        un = unit_of<MODE, KIND, WB, true>(g, work, j + g.P);
        copy_list<KIND>(g, un, list_u(1), wave, lane);
    }
    wait_vm_lgkm<0>();
    slot_barrier();
    Copier<MODE, KIND, WEIGHTS, WB> cp;
    cp.setup(g, u, list(0), wave, lane);
    int m = 0;       // this unit's number
    int with = 0;    // whether the last stage copied came with scales
    int at = 0;      // slot of the stage being computed
    int to = 0;      // slot of the next copies
    auto next_unit = [&]() {
        if (cp.st == cp.KT) {
            if (more) cp.setup(again(), un, list(m + 1), wave, opaque_v(lane));
            else cp.nothing();
        }
        with = cp.scaled();
    };
    auto copy_next = [&]() {
        next_unit();
        cp.stage(lds_u + (uint32_t)to * GE::kSlot, lds_u + GE::kScale0 + (uint32_t)to * GE::kScale, wave, lane);
        to = to + 1 == GE::kSlots ? 0 : to + 1;
    };
    for (int i = 0; i < GE::kAhead; ++i) copy_next();

    for (;;) {
        f32x16 acc[GE::TB][2];
#pragma unroll
        for (int b = 0; b < GE::TB; ++b)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[b][q][v] = 0.0f;
        Unit u2 = un;
        bool more2 = false;
        const int KT = GE::stream_stages(u.KT);
        int cut = -1;  // the stage of 128 values only, in the order of the stages computed
        if constexpr (GE::kPanels == 2) {
            const Gemm ga = again();
            const int K = MODE == kGateUp ? ga.H : ga.F;
            if (K % (2 * kTK)) {
                cut = stages<KIND, WB>(K) - 1 - u.k0 - u.rot;
                cut = uni(cut < 0 ? cut + u.KT : cut);
            }
        }
        uint32_t wnext[2][2], tnext[2][GE::TB];  // [panel]: the odd stage's scales, from the even one
        for (int s = 0; s < KT; ++s) {
            // this stage landed in this wave: the copies of the kAhead - 1
            // stages after it may be out (a list or stores among them only
            // make the wait longer)
            static_assert(GE::kPanels == 1 || GE::kAhead <= 2, "the stage after this one is the last copied");
            if (GE::kPanels == 2 && GE::kAhead == 2 && !uni(with)) wait_vm_lgkm<GE::kPerStage - 2>();
            else wait_vm_lgkm<(GE::kAhead - 1) * GE::kPerStage>();
            slot_barrier();  // ... in every wave; the slot of the stage before is free
            if (s == 0) {
                // the unit after next: its list goes to the place of the list
                // of the unit before this one, whose epilogue is done; it
                // lands before the first stage of the next unit does, whose
                // copies follow it
                more2 = j + 2 * P < end;
                if (more2) {
                    const Gemm ga = again();
                    u2 = unit_of<MODE, KIND, WB>(ga, work, j + 2 * P);
                    copy_list<KIND>(ga, u2, list_u(m + 2), wave, lane);
                }
            }
            // (4-bit weights: the rows' and the scales' copies go out behind the reads of this
            // stage's operands: 128 experts of 16, 50 and 100 rows of 4096 x 1536, gate/up and
            // down, 252 -> 246, 360 -> 333 and 386 -> 370 us. They are written among the
            // products, but do not run beside them: scales has a branch, and the compiler puts
            // every product behind it. Written in front of all products, in the order that
            // runs, they took 1 % longer at 50 rows, 340 -> 346 us, and as long at 16 and 100)
            const uint32_t cslot = lds_u + (uint32_t)to * GE::kSlot, csslot = lds_u + GE::kScale0 + (uint32_t)to * GE::kScale;
            auto pieces = [&](auto from, auto count) {
                unrolled([&](auto i) { cp.template piece<decltype(from)::value + decltype(i)::value>(cslot, csslot, wave, lane); },
                         std::make_integer_sequence<int, decltype(count)::value>{});
            };
            if constexpr (GE::kPanels == 2) {
                next_unit();
                to = to + 1 == GE::kSlots ? 0 : to + 1;
                pieces(Number<0>{}, Number<GE::kWCopies>{});
            } else {
                copy_next();
            }
            const char* slot = lds + at * GE::kSlot;
            const char* ssl = lds + GE::kScale0 + at * GE::kScale;
            at = at + 1 == GE::kSlots ? 0 : at + 1;
            uint32_t wnow[2][2], tnow[2][GE::TB];
            if constexpr (GE::kPanels == 2) {
                const bool odd = (u.k0 + s) & 1;
                if (odd && s > 0) {
                    // (past the unit's last stage they are the next rows', maybe NaN, on codes of 0)
                    const uint32_t keep = s < u.KT ? ~0u : 0u;
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) wnow[p][q] = wnext[p][q] & keep;
#pragma unroll
                        for (int b = 0; b < GE::TB; ++b) tnow[p][b] = tnext[p][b] & keep;
                    }
                } else {
                    auto read = [&](int row, uint32_t& n0, uint32_t& n1, uint32_t& x0, uint32_t& x1) {
                        const u32x4 w = *reinterpret_cast<const u32x4*>(ssl + row * 16);
                        n0 = odd ? w[2] : w[0];
                        n1 = odd ? w[3] : w[1];
                        x0 = w[2];
                        x1 = w[3];
                    };
#pragma unroll
                    for (int q = 0; q < 2; ++q) read(GE::wrow(wn, q) + fr, wnow[0][q], wnow[1][q], wnext[0][q], wnext[1][q]);
#pragma unroll
                    for (int b = 0; b < GE::TB; ++b) read(kTN + 32 * b + fr, tnow[0][b], tnow[1][b], tnext[0][b], tnext[1][b]);
                }
            }
            if constexpr (GE::kPanels == 2) {
                constexpr int S = kSplit ? 2 : 1, kMfmas = 4 * GE::TB * 2 * S, kLeft = GE::kACopies + 1;
                const char *const weights = slot + GE::kA;
                i32x8 wf[4][2], tf[4][GE::TB], low;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c0 = ((4 * (k % 2) + half) ^ swz(fr)) * 16, c1 = ((4 * (k % 2) + 2 + half) ^ swz(fr)) * 16;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        wf[k][i] = wfrag<4>(weights + (GE::wrow(wn, i) + fr) * GE::kWRow + ((2 * k + half) ^ swz(fr)) * 16, weights);
#pragma unroll
                    for (int b = 0; b < GE::TB; ++b) {
                        const char* t = slot + k / 2 * (GE::kRows * kTK) + (32 * b + fr) * 128;
                        tf[k][b] = frag(t + c0, t + c1);
                    }
                }
                // this lane's blocks: bytes 0 and 2 of the words, 1 and 3 in the upper lanes
                // (past a row's end the scales are the next row's, maybe NaN, on codes of 0)
                const uint32_t keep = s == cut ? 0u : ~0u;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) wnow[p][q] = (p ? wnow[p][q] & keep : wnow[p][q]) >> 8 * half;
#pragma unroll
                    for (int i = 0; i < GE::TB; ++i) tnow[p][i] = (p ? tnow[p][i] & keep : tnow[p][i]) >> 8 * half;
                }
                __builtin_amdgcn_sched_barrier(0);
                unrolled([&](auto n_tag) {
                    constexpr int n = decltype(n_tag)::value, q = n % 2, sp = n / 2 % S, b = n / (2 * S) % GE::TB;
                    constexpr int k = n / (2 * S * GE::TB), p = k / 2;
                    if constexpr (kSplit && n % (2 * S) == 0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int up = (int)upper_codes((uint32_t)tf[k][b][i]);
                            low[i] = tf[k][b][i] ^ up;
                            tf[k][b][i] = up;
                        }
                    }
                    acc[b][q] = mfma<4, 2 * (k % 2)>(wf[k][q], sp ? low : tf[k][b], acc[b][q], wnow[p][q], tnow[p][b]);
                    constexpr int from = n * kLeft / kMfmas, upto = (n + 1) * kLeft / kMfmas;
                    if constexpr (upto > from) {
                        __builtin_amdgcn_sched_barrier(0);
                        pieces(Number<GE::kWCopies + from>{}, Number<upto - from>{});
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }, std::make_integer_sequence<int, kMfmas>{});
            } else {
                // 128 values of K: the four blocks' scales of each weight and row
                const char *const rows = slot, *const weights = slot + GE::kA;
                uint32_t ws[2], ts[GE::TB];
#pragma unroll
                for (int q = 0; q < 2; ++q) ws[q] = *reinterpret_cast<const uint32_t*>(ssl + (GE::wrow(wn, q) + fr) * 4);
#pragma unroll
                for (int b = 0; b < GE::TB; ++b) ts[b] = *reinterpret_cast<const uint32_t*>(ssl + (kTN + 32 * b + fr) * 4);
                if constexpr (kWide) {
                    auto block = [&](auto b_tag) {  // 32 values of K, 16 per half of the wave
                        constexpr int B = decltype(b_tag)::value;
                        const int c = ((2 * B + half) ^ swz(fr)) * 16;
                        Bf16x16 wf[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            wf[q] = widen<B>(*reinterpret_cast<const u32x4*>(weights + (GE::wrow(wn, q) + fr) * GE::kWRow + c), ws[q]);
#pragma unroll
                        for (int b = 0; b < GE::TB; ++b) {
                            const Bf16x16 tf = widen<B>(*reinterpret_cast<const u32x4*>(rows + (32 * b + fr) * 128 + c), ts[b]);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                acc[b][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[q].lo, tf.lo, acc[b][q], 0, 0, 0);
                                acc[b][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[q].hi, tf.hi, acc[b][q], 0, 0, 0);
                            }
                        }
                    };
                    block(std::integral_constant<int, 0>{});
                    block(std::integral_constant<int, 1>{});
                    block(std::integral_constant<int, 2>{});
                    block(std::integral_constant<int, 3>{});
                } else {
                    // this lane's blocks: bytes 0 and 2 of the word, 1 and 3 in the upper lanes
#pragma unroll
                    for (int q = 0; q < 2; ++q) ws[q] >>= 8 * half;
#pragma unroll
                    for (int b = 0; b < GE::TB; ++b) ts[b] >>= 8 * half;
                    auto kstep = [&](auto kk_tag) {
                        constexpr int KK = decltype(kk_tag)::value;
                        const int c0 = ((4 * KK + half) ^ swz(fr)) * 16, c1 = ((4 * KK + 2 + half) ^ swz(fr)) * 16;
                        i32x8 wf[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const char* w = weights + (GE::wrow(wn, q) + fr) * GE::kWRow;
                            wf[q] = frag(w + c0, w + c1);
                        }
#pragma unroll
                        for (int b = 0; b < GE::TB; ++b) {
                            const char* t = rows + (32 * b + fr) * 128;
                            const i32x8 tf = frag(t + c0, t + c1);
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                acc[b][q] = mfma<8, 2 * KK>(wf[q], tf, acc[b][q], ws[q], ts[b]);
                        }
                    };
                    kstep(std::integral_constant<int, 0>{});
                    kstep(std::integral_constant<int, 1>{});
                }
            }
        }
        drain();
        const Gemm ga = again();
        if (u.pidx >= 0) {
#pragma unroll
            for (int b = 0; b < GE::TB; ++b) store_part<MODE, KIND>(ga, u, b, acc[b], wave, opaque_v(lane));
        } else {
#pragma unroll
            for (int b = 0; b < GE::TB; ++b) finish<MODE, KIND>(ga, u, b, acc[b], list(m), wave, opaque_v(lane));
        }
        if (!more) break;
        u = un;
        un = u2;
        more = more2;
        j += P;
        ++m;
    }
}

// ------------------------------------------------------- 256-row tiles --
// A stage is 32 MFMAs of 64 cycles a wave on 64 KB of copies and 128 KB of LDS
// reads, so the three have to overlap throughout:
//   first half of stage s: the products of its first 64 values of K, the reads
//     of the second 64, and the copies of the first 128 weight rows of stage
//     s + 2, into the fifth unit of the ring, which no stage in use holds;
//   one barrier: stage s's fragments are all in registers (its units and its
//     row slot are free) and stage s + 1 has landed (each wave waits for its
//     own copies but the four it just issued);
//   second half: the other products, the copies of the other weight rows and of
//     the rows of stage s + 2, and the reads of stage s + 1's first 64 values.
// (All copies in one half took 2.5 us a stage: the waves that issue them wait
// for the copy path, and their MFMAs with them.)
//
// Measured in a stream of calls, once the clock has settled (counters of cycles
// and of time read inside the kernel; tile ends included in the stages): 8 experts
// of 512 rows of 4096 x 14336, gate/up, 3230 cycles at 1.81 GHz = 1.78 us a stage, 63 %
// of them products; the same with codes random in every bit 3150 at 1.67 GHz; 4094
// rows of them unevenly, 3090 at 1.95 GHz (58 %). In the first calls after idle the
// clock is lower (1.5 to 1.75 GHz) and a stage has fewer cycles (2800 to 3180). So it
// is two things: power holds the clock below the 2.2 GHz of the short-K layers, and what does not
// follow the clock, a stage's 64 KB of copies (37 GB/s a CU here, 52 to 56 where a
// CU only copies), overlaps the products in part only. Fewer scalar instructions
// beside the products (the ring's units of 128 rows for 32) took 8 experts of 512 rows
// of 4096 x 14336 from 519 to 484 us (gate/up) and from 245 to 232 us (down), in calls
// of random codes at the lower clock.
//
// One wave's vector memory instruction costs as much for 64 lines of 16 bytes as
// for a kilobyte in 8: copies of 4 bytes of scales a stage for each of the 512
// rows cost 16 % of the time. They come in groups of up to four stages instead
// (16 bytes a row): a group waits in LDS, is read into registers in the last
// stage of the group before it, and its place is filled again in the stage
// after.

// The product of a half stage after which fragment id (0..3 weights, 4..7 rows)
// of the other half is read: the weights first, a row block once the same
// block of this half has been used (it can take its registers), the last ones
// early enough to arrive before the half ends.
__host__ __device__ constexpr int read_at(int id, int products)
{
    return id < 4 ? (id < products ? id : products - 1)
                  : 4 * (id - 3) < products - 3 ? 4 * (id - 3) : products - 3;
}

// Groups of scales of a workgroup's units of kind 0, in the order of the
// stream: stages a .. a + len of K, loaded from stage a - skip on (the last 16
// bytes of a row, near its end). No group but a whole unit has one stage.
template <int MODE>
struct ScaleStream {
    uint32_t asoff;
    int e, n0, x0, at, left, len, skip;

    __device__ __forceinline__ void setup(const Gemm& g, const Unit& u, const int32_t* list, int wave, int lane)
    {
        const int KS = (MODE == kGateUp ? g.H : g.F) / moe::kMxBlock;
        e = u.e;
        n0 = u.n0;
        x0 = MODE == kGateUp ? 0 : u.x0;
        at = u.k0 + u.rot;
        left = Geo<MODE, 0, 8>::stream_stages(u.KT);
        const int r = 64 * wave + lane;
        uint32_t off = (MODE == kGateUp ? (uint32_t)list[r] : (uint32_t)r) * (uint32_t)KS;
        asm volatile("" : "+v"(off));  // (as in Copier)
        asoff = r < u.rows ? off : kZeroRow;
    }
    __device__ __forceinline__ void nothing()  // the last unit's scales again, for no one
    {
        at = 0;
        left = 0x7fffffff;
    }
    // copies the next group
    __device__ __forceinline__ void copy(const Gemm& g, uint32_t lds, int wave, int lane)
    {
        const int K = MODE == kGateUp ? g.H : g.F, KS = K / moe::kMxBlock, wrows = MODE == kGateUp ? g.F : g.H;
        const int KT_all = K / kTK, from = min(at, KT_all - 4);
        skip = at - from;
        len = min(4 - skip, left);
        if (left - len == 1 && len > 1) --len;
        const int r = 64 * wave + lane;
        const uint32_t wsoff = (uint32_t)(MODE == kGateUp ? n0 + (r & 127) : min(n0 + r, wrows - 1)) * (uint32_t)KS;
        const uint8_t* s = MODE == kGateUp && wave >= 2 ? g.s1 : g.s0;
        copy16(buffer_of(s + (size_t)e * wrows * KS, kCopyRange), wsoff, from * 4, lds + wave * 1024);
        copy16(buffer_of(g.as + (size_t)x0 * KS, kCopyRange), asoff, from * 4, lds + kTN * 16 + wave * 1024);
        at += len;
        if (at == KT_all) at = 0;  // (only where the unit began past 0)
        left -= len;
    }
};

template <int MODE, int WB>
__device__ __forceinline__ void big_tiles(const Gemm& g, char* lds)
{
    using GE = Geo<MODE, 0, WB>;
    const KindWork work = work_of<MODE, WB>(g, 0);
    const int end = work.count;
    // Round r's tile at position p goes to slot p + r: tails lie between whole
    // tiles at regular distances, and no slot should get only the one or the
    // other.
    auto unit_at = [](const Gemm& g, int r) {
        const int b = blockIdx.x, slot = b % 8 * (g.P / 8) + b / 8;
        return r * g.P + uni((slot - r % g.P + g.P) % g.P);
    };
    const int units = uni(end / g.P + (unit_at(g, end / g.P) < end));  // this workgroup's
    if (units == 0) return;

    const int tid = threadIdx.x, wave = uni(tid >> 6), lane = tid & 63;
    const int fr = lane & 31, half = lane >> 5, wm = wave >> 1, wn = wave & 1;
    const uint32_t lds_u = (uint32_t)(uintptr_t)lds;
    auto list = [&](int m) { return reinterpret_cast<const int32_t*>(lds + GE::kList0 + m % 3 * GE::kRows * 4); };
    auto list_u = [&](int m) { return lds_u + GE::kList0 + m % 3 * GE::kRows * 4; };

    // the units ahead wait in LDS, each wave's own copies: scalar registers held
    // across a tile's stages would be spilled
    auto keep = [&](int m, const Unit& u) {
        int4* p = reinterpret_cast<int4*>(lds + GE::kKept0) + (wave * 3 + m % 3) * 2;
        p[0] = make_int4(u.e, u.n0, u.rows, u.x0);
        p[1] = make_int4(u.k0, u.KT, u.pidx, u.rot);
    };
    auto kept = [&](int m) {
        const int4* p = reinterpret_cast<const int4*>(lds + GE::kKept0) + (wave * 3 + m % 3) * 2;
        const int4 a = p[0], b = p[1];
        return Unit{uni(a.x), uni(a.y), uni(a.z), uni(a.w), uni(b.x), uni(b.y), uni(b.z), uni(b.w), 0};
    };
    Unit u = unit_of<MODE, 0, WB, true>(g, work, unit_at(g, 0));
    copy_list<0>(g, u, list_u(0), wave, lane);
    if (units > 1) {
        const Unit un = unit_of<MODE, 0, WB, true>(g, work, unit_at(g, 1));
        keep(1, un);
        copy_list<0>(g, un, list_u(1), wave, lane);
    }
    wait_vm_lgkm<0>();
    slot_barrier();
    Copier<MODE, 0, kKept, WB> cp;
    cp.setup(g, u, list(0), wave, lane);
    int m = 0, odd = 0;  // this unit's number; parity of the stage being computed
    constexpr int kEarly = GE::kWCopies / 2;  // weight copies in a stage's first half (one unit)
    constexpr int kLate = GE::kACopies + GE::kWCopies - kEarly;
    // the copies move on to the next unit
    auto follow = [&]() {
        if (cp.st == cp.KT) {
            if (m + 1 < units) cp.setup(again(), kept(m + 1), list(m + 1), wave, opaque_v(lane));
            else cp.nothing();
        }
    };
    auto slot_u = [&](int n) { return lds_u + (uint32_t)n * GE::kSlot; };
    // ring units: the stage being computed holds units wat and wat + 1, the
    // next one the two after them, and so on
    auto wrap = [&](int x) { return x >= GE::kUnits ? x - GE::kUnits : x; };
    int wat = 0;
    auto unit_u = [&](int unit, int i) { return lds_u + GE::kUnit0 + (uint32_t)unit * GE::kUnit + (uint32_t)(i % kEarly) * 4096u; };

    i32x8 wf[2][4], tf[2][4];
    // Scales of this stage and the rest of its group: the lane's two bytes of
    // each stage (blocks 0 and 2 of the four; 1 and 3 in the upper lanes),
    // this stage's in the lowest.
    u32x2 ws[4], ts[4];
    // fragment addresses: chunk c of row r is slot chunk c ^ swz(r); of a
    // lane's four chunks (half, half + 2, + 4, + 6) the others differ from
    // the first in address bits 5 and 6 (4-bit weights: of two, half and half +
    // 2, in bit 5)
    const uint32_t fc = (uint32_t)((half ^ swz(fr)) * 16);
    const uint32_t wfa = (uint32_t)(GE::kUnit0 + ((MODE == kGateUp ? wn * 64 : 0) + fr) * GE::kWRow) +
                         (WB == 8 ? fc : (uint32_t)((half ^ swz4(fr)) * 16));
    const uint32_t tfa = (uint32_t)((wm * 32 + fr) * 128) + fc;
    // fragment id (0..3 weights, 4..7 rows) of the stage in row slot n whose
    // weights start at unit w0 of the ring
    auto read = [&](int n, int w0, int kk, int id) {
        if (id < 4) {
            // gate/up: blocks 0, 1 in the stage's first unit (gate), 2, 3 in the
            // second; down: all four in unit wn
            const int unit = MODE == kGateUp ? (id < 2 ? w0 : wrap(w0 + 1)) : wn == 0 ? w0 : wrap(w0 + 1);
            const int o = (MODE == kGateUp ? id % 2 : id) * 32 * GE::kWRow;
            const uint32_t at = (wfa ^ (uint32_t)(GE::kWRow / 2 * kk)) + (uint32_t)unit * GE::kUnit;
            wf[kk][id] = wfrag<WB>(lds + at + o, lds + (at ^ 32u) + o);
        } else {
            const uint32_t at = (tfa ^ (uint32_t)(64 * kk)) + (uint32_t)n * GE::kSlot;
            const int o = (id - 4) * 8192;
            tf[kk][id - 4] = frag(lds + at + o, lds + (at ^ 32u) + o);
        }
    };
    // the group that waits in LDS
    const uint32_t sel = half ? 0x07050301u : 0x06040200u;
    auto pack = [&](const u32x4& v) {
        return u32x2{__builtin_amdgcn_perm(v[1], v[0], sel), __builtin_amdgcn_perm(v[3], v[2], sel)};
    };
    auto read_group = [&](u32x2* w, u32x2* t, int skip) {
        const char* p = lds + GE::kScale0;
        u32x4 a[4], b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            a[q] = *reinterpret_cast<const u32x4*>(p + (GE::wrow(wn, q) + fr) * 16);
            b[q] = *reinterpret_cast<const u32x4*>(p + (kTN + (2 * q + wm) * 32 + fr) * 16);
        }
        __builtin_amdgcn_sched_barrier(0);  // all reads in flight together
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = pack(a[q]);
            t[q] = pack(b[q]);
        }
        if (skip > 0)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                w[q] = __builtin_bit_cast(u32x2, __builtin_bit_cast(uint64_t, w[q]) >> (16 * skip));
                t[q] = __builtin_bit_cast(u32x2, __builtin_bit_cast(uint64_t, t[q]) >> (16 * skip));
            }
    };
    // the next stage's scales: the next of the group, or the next group's
    // first (selected: a branch here would be one below the products)
    auto next_scale = [](u32x2& v, const u32x2& group, bool refill) {
        const uint64_t next = __builtin_bit_cast(uint64_t, v) >> 16;
        v = __builtin_bit_cast(u32x2, refill ? __builtin_bit_cast(uint64_t, group) : next);
    };
    // the scales' copies move on to the next unit and copy its next group
    ScaleStream<MODE> sc;
    auto copy_group = [&](int lists) {
        if (sc.left == 0) {
            if (lists + 1 < units) sc.setup(again(), kept(lists + 1), list(lists + 1), wave, opaque_v(lane));
            else sc.nothing();
        }
        sc.copy(again(), lds_u + GE::kScale0, wave, opaque_v(lane));
    };
    sc.setup(g, u, list(0), wave, lane);
    sc.copy(again(), lds_u + GE::kScale0, wave, opaque_v(lane));
    int glen = sc.len;         // stages of this group that are left
    const int gskip = sc.skip;
    for (int n = 0; n < 2; ++n) {
        follow();
#pragma unroll
        for (int i = 0; i < GE::kWCopies; ++i) cp.template weight<false>(i, unit_u(2 * n + i / kEarly, i), wave);
#pragma unroll
        for (int i = 0; i < GE::kACopies; ++i) cp.row(i, slot_u(n), wave);
        ++cp.st;
    }
    wait_vm_lgkm<0>();
    slot_barrier();
#pragma unroll
    for (int id = 0; id < 8; ++id) read(0, 0, 0, id);
    read_group(ws, ts, gskip);
    wait_vm_lgkm<0>();
    slot_barrier();
    copy_group(0);
    int nlen = sc.len, nskip = sc.skip;  // the group in LDS
    bool refill = false;                 // it has been read: its place is free

    // One unit whose rows fill NB token blocks of each wave (32 rows of every
    // 64): its stages and its epilogue.
    auto run = [&](auto nb_tag) {
        constexpr int NB = decltype(nb_tag)::value, kM = 4 * NB;  // products per half stage
        f32x16 acc[NB][4];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][q][v] = 0.0f;
        const int KT = GE::stream_stages(u.KT);
        for (int s = 0; s < KT; ++s) {
            // (no branch below this: the compiler would move the first half's
            // products behind it, next to their uses)
            if (s == 1) {
                // the unit after next: its list goes to the place of the list
                // of the unit before this one, whose epilogue every wave left
                // before stage 0's barrier
                if (m + 2 < units) {
                    const Gemm ga = again();
                    const Unit u2 = unit_of<MODE, 0, WB>(ga, work_of<MODE, WB>(ga, 0), unit_at(ga, m + 2));
                    keep(m + 2, u2);
                    copy_list<0>(ga, u2, list_u(m + 2), wave, opaque_v(lane));
                }
            }
            follow();
            // the next group's scales; what they hold in other stages is not used
            u32x2 wsn[4], tsn[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) asm("" : "=v"(wsn[q]), "=v"(tsn[q]));
            if (refill) {  // read by every wave before the last barrier
                copy_group(m);
                nlen = sc.len;
                nskip = sc.skip;
            }
            refill = glen == 1;
            if (refill) {  // the next stage starts the group in LDS
                read_group(wsn, tsn, nskip);
            }
            const int wnext = wrap(wat + 2), wcopy = wrap(wnext + 2), wcopy1 = wrap(wcopy + 1);
#pragma unroll
            for (int q = 0; q < kM; ++q) {
                acc[q >> 2][q & 3] = mfma<WB, 0>(wf[0][q & 3], tf[0][q >> 2], acc[q >> 2][q & 3], ws[q & 3][0], ts[q >> 2][0]);
                // this half's share of the reads (NB row blocks) and copies
#pragma unroll
                for (int z = 0; z < 4 + NB; ++z)
                    if (read_at(z, kM) == q) read(odd, wat, 1, z);
#pragma unroll
                for (int z = q * kEarly / kM; z < (q + 1) * kEarly / kM; ++z) cp.template weight<false>(z, unit_u(wcopy, z), wave);
                __builtin_amdgcn_sched_barrier(0);
            }
            wait_vm_lgkm<kEarly>();
            slot_barrier();  // the next stage has landed, and this one's slots are free
            const uint32_t sl = slot_u(odd);
#pragma unroll
            for (int q = 0; q < kM; ++q) {
                acc[q >> 2][q & 3] = mfma<WB, 1>(wf[1][q & 3], tf[1][q >> 2], acc[q >> 2][q & 3], ws[q & 3][0], ts[q >> 2][0]);
#pragma unroll
                for (int z = q * kLate / kM; z < (q + 1) * kLate / kM; ++z) {
                    if (z < GE::kACopies) cp.row(z, sl, wave);
                    else if (z - GE::kACopies < GE::kWCopies - kEarly)
                        cp.template weight<false>(kEarly + z - GE::kACopies, unit_u(wcopy1, z), wave);
                }
#pragma unroll
                for (int z = 0; z < 8; ++z)
                    if (read_at(z, kM) == q) read(odd ^ 1, wnext, 0, z);
                // scales that no product of this stage needs any more
                if (q % 4 == 3 && q < kM - 1) next_scale(ts[q >> 2], tsn[q >> 2], refill);
                if (q >= kM - 4) next_scale(ws[q - (kM - 4)], wsn[q - (kM - 4)], refill);
                if (q == kM - 1)
#pragma unroll
                    for (int i = NB - 1; i < 4; ++i) next_scale(ts[i], tsn[i], refill);
                __builtin_amdgcn_sched_barrier(0);
            }
            ++cp.st;
            wat = wnext;
            odd ^= 1;
            glen = refill ? nlen : glen - 1;
        }
        drain();
        const Gemm ga = again();
        if (u.pidx >= 0) {
#pragma unroll
            for (int i = 0; i < NB; ++i) store_part<MODE, 0>(ga, u, i, acc[i], wave, opaque_v(lane));
        } else {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                finish<MODE, 0>(ga, u, i, acc[i], list(m), wave, opaque_v(lane));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    for (;;) {
        if (u.rows > 192) run(std::integral_constant<int, 4>{});
        else if (u.rows > 128) run(std::integral_constant<int, 3>{});
        else if (u.rows > 64) run(std::integral_constant<int, 2>{});
        else run(std::integral_constant<int, 1>{});
        if (++m == units) break;
        u = kept(m);
    }
}

// BASE: kind of an expert's whole tiles (mx_base)
template <int MODE, int BASE, int WB>
__global__ __launch_bounds__(kThreads, 1) void gemm_mx_kernel(const Gemm g)
{
    __shared__ __attribute__((aligned(1024))) char lds[kLds<WB>];
    const int b = blockIdx.x;
    const int slot_id = b % 8 * (g.P / 8) + b / 8;
    if constexpr (BASE == 0) big_tiles<MODE, WB>(g, lds);
    ring_tiles<MODE, 1, BASE == 0 ? kStreamed : kByExpert, WB>(g, lds, slot_id);
    ring_tiles<MODE, 2, kStreamed, WB>(g, lds, slot_id);
    ring_tiles<MODE, 3, kStreamed, WB>(g, lds, slot_id);
}

// Whether a launch may cut tiles along K: not where the rows alone make
// kSplitRounds rounds of tiles, whatever their experts (the fixup then need not
// be launched, 5 us), nor where K has no two parts. (Counted in stages of 128 values: small
// tiles of 4-bit weights, of stages of 256, are not cut below K = 1920, and where K is 1024
// and more the fixup is launched for them all the same, and finds nothing.)
inline bool may_split(const moe_shape_t& s, int mode, int P)
{
    const int64_t N = (int64_t)s.T * s.k, ntn = mode == kGateUp ? s.F / (kTN / 2) : (s.H + kTN - 1) / kTN;
    const int KT = (mode == kGateUp ? s.H : s.F) / kTK, top = mx_rows(moe::mx_base(s));
    return KT >= 2 * moe::kMxMinStages && (N + top - 1) / top * ntn < (int64_t)kSplitRounds * P;
}

// Adds the K-parts of split tiles in order: workgroup (tile, token block) of
// a kind, its waves as the tile's.
//
// fix_items: the most (tile, block) pairs of a kind that the launch can have
// to finish: fewer than P tiles are split, and no more than it can have at
// all. (An expert can hold every assignment, not one of each token only: ids
// that name it twice are flagged by the count, and computed.)
inline int fix_items(const moe_shape_t& s, int mode, int kind, int P)
{
    const int base = moe::mx_base(s), tb = kind == 0 ? 4 : mx_rows(kind) / 32;
    if (kind < base) return 0;
    if (kind < kMxKinds - 1 && (int64_t)s.T * s.k <= mx_rows(kind + 1)) return 0;
    const int ntn = mode == kGateUp ? s.F / (kTN / 2) : (s.H + kTN - 1) / kTN;
    const int64_t tiles = moe::mx_tiles(s, kind) * ntn;
    return (int)(tiles < P ? tiles : P) * tb;
}

template <int MODE, int KIND, int WB>
__device__ __forceinline__ void fix_tile(const Gemm& g, int item)
{
    using GE = Geo<MODE, KIND, 8>;
    const KindWork w = work_of<MODE, WB>(g, KIND);
    const int t = item / GE::TB, i = item % GE::TB;
    if (w.S == 1 || t >= w.L) return;
    Unit u;
    tile_by_wave<MODE, KIND>(g, w.full + t, u);
    const int wave = uni((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave / GE::WN;
    if ((i * GE::WM + wm) * 32 >= u.rows) return;
    f32x16 acc[GE::WBL];
#pragma unroll
    for (int j = 0; j < GE::WBL; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][v] = 0.0f;
    const int last = (i * GE::WM + wm) * 32 + (lane & 31) < u.rows ? w.S : 0;  // padding rows have no parts
    for (int p = 0; p < last; ++p)
#pragma unroll
        for (int j = 0; j < GE::WBL; ++j) {
            const float4* src = part_at<MODE, KIND>(g, p * w.L + t, wave, i, j, lane);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 v = src[q * 64];
                acc[j][4 * q] += v.x;
                acc[j][4 * q + 1] += v.y;
                acc[j][4 * q + 2] += v.z;
                acc[j][4 * q + 3] += v.w;
            }
        }
    finish<MODE, KIND>(g, u, i, acc, g.vrow + u.x0, wave, lane);
}

struct FixGrid {
    int end[kMxKinds];
};

template <int MODE, int WB>
__global__ __launch_bounds__(kThreads) void mx_fixup_kernel(const Gemm g, const FixGrid f)
{
    const int b = blockIdx.x;
    if (b < f.end[0]) fix_tile<MODE, 0, WB>(g, b);
    else if (b < f.end[1]) fix_tile<MODE, 1, WB>(g, b - f.end[0]);
    else if (b < f.end[2]) fix_tile<MODE, 2, WB>(g, b - f.end[1]);
    else fix_tile<MODE, 3, WB>(g, b - f.end[2]);
}

template <int MODE, int WB>
hipError_t launch_fixup(const Gemm& g, const moe_shape_t& s, hipStream_t st)
{
    if (!g.split) return hipSuccess;
    FixGrid f;
    int n = 0;
    for (int k = 0; k < kMxKinds; ++k) f.end[k] = n += fix_items(s, MODE, k, g.P);
    if (n == 0) return hipSuccess;
    mx_fixup_kernel<MODE, WB><<<n, kThreads, 0, st>>>(g, f);
    return hipGetLastError();
}

// One workgroup per CU, a multiple of 8 (as many on every XCD), at most what
// the partial tiles' workspace is sized for.
int persistent_grid()
{
    static const int grid = [] {
        int dev = 0, cus = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            cus = moe::kGemmMaxGrid;
        const int g = cus >= 8 ? cus / 8 * 8 : 8;
        return g < moe::kGemmMaxGrid ? g : moe::kGemmMaxGrid;
    }();
    return grid;
}

template <int WB>
hipError_t launch(const moe_shape_t& s, const void* a, const void* a_s, const int32_t* plan, const MoeMxWeights& w,
                  void* y, char* ws, hipStream_t st)
{
    const int N = s.T * s.k, base = moe::mx_base(s);
    if (N == 0) return hipSuccess;
    const moe::MxWsLayout W = moe::mx_ws_layout(s);
    int32_t* sched = reinterpret_cast<int32_t*>(ws + W.sched);
    int32_t* vrow = reinterpret_cast<int32_t*>(ws + W.vrow);
    mx_schedule_kernel<<<(N + kThreads - 1) / kThreads, kThreads, 0, st>>>(s.E, s.R, N, base, plan, sched, vrow);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    Gemm g;
    g.E = s.E;
    g.H = s.H;
    g.F = s.F;
    g.P = persistent_grid();
    g.N = N;
    g.sched = sched;
    g.vrow = vrow;
    g.h = reinterpret_cast<uint8_t*>(ws + W.h);
    g.hs = reinterpret_cast<uint8_t*>(ws + W.hs);
    g.y = static_cast<uint16_t*>(y);
    for (int k = 0; k < kMxKinds; ++k) g.part[k] = reinterpret_cast<float*>(ws + W.part[k]);
    g.ntn = s.F / (kTN / 2);
    g.split = may_split(s, kGateUp, g.P);
    g.a = static_cast<const uint8_t*>(a);
    g.as = static_cast<const uint8_t*>(a_s);
    g.w0 = w.gate;
    g.s0 = w.gate_s;
    g.w1 = w.up;
    g.s1 = w.up_s;
    (base == 0 ? gemm_mx_kernel<kGateUp, 0, WB> : gemm_mx_kernel<kGateUp, 1, WB>)<<<g.P, kThreads, 0, st>>>(g);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = launch_fixup<kGateUp, WB>(g, s, st)) != hipSuccess) return e;
    g.ntn = (s.H + kTN - 1) / kTN;
    g.split = may_split(s, kDown, g.P);
    g.a = g.h;
    g.as = g.hs;
    g.w0 = w.down;
    g.s0 = w.down_s;
    g.w1 = g.s1 = nullptr;
    (base == 0 ? gemm_mx_kernel<kDown, 0, WB> : gemm_mx_kernel<kDown, 1, WB>)<<<g.P, kThreads, 0, st>>>(g);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    return launch_fixup<kDown, WB>(g, s, st);
}

}  // namespace

hipError_t moe_launch_grouped_gemm_mx(const moe_shape_t& s, const void* a, const void* a_s,
                                      const int32_t* plan, const MoeMxWeights& w, void* y,
                                      char* ws, hipStream_t st)
{
    return launch<8>(s, a, a_s, plan, w, y, ws, st);
}

hipError_t moe_launch_grouped_gemm_mx4(const moe_shape_t& s, const void* a, const void* a_s,
                                       const int32_t* plan, const MoeMxWeights& w, void* y,
                                       char* ws, hipStream_t st)
{
    return launch<4>(s, a, a_s, plan, w, y, ws, st);
}
