// few.hip -- a whole MoE layer for up to 32 tokens (moe_few_layer).
//
//   logits = x Wr^T; top-k of logits + bias; w = softmax of the chosen logits;
//   out = sum_j w_j Wd (silu(Wg x) * (Wu x)) (+ the shared expert).
//
// Bound by the live experts' weights, each read once (few_two_tiles says where an
// expert with more than 16 rows reads them again). A step is 16 weight rows
// of two streams (gate and up; in the down projection, two neighbours) times up
// to 16 rows of one expert, or 32, on v_mfma_f32_16x16x32_bf16 (codes are widened to
// bf16, exactly but at the ends of the scales' range); the rows' values stay in registers from step to step. The eight
// waves of a workgroup share K; each brings its own weights through a ring of
// copies in LDS that runs across steps (12 to 14 KB in flight a wave), and their
// sums meet in LDS. A workgroup takes a run of neighbouring steps, so that it
// changes its expert rarely.
//
// The copies are what the ring is for: 64 lanes that load operands straight into
// registers touch 64 places of 16 bytes (lanes of a row are 16 apart), each a
// lookup of its own in the cache in front, which was busy two thirds of the time
// that way; a copy's lanes read 64 or 128 bytes of a row in turn.
//
// h = silu(g) u is kept as two bf16 (value and remainder, see two_bf16), so that it
// carries 16 bits into the down projection; its sums are kept in fp32 for each assignment
// and added in j order.
//
// Measured (us and TB/s of weights, two layers in turn): one token, 8 of 128 experts,
// 4096 x 1536, bf16: scores 4.7, gate/up 36 (5.5), down 19 (5.2), combine 4.6; five
// tokens, top-2 of 8, 4096 x 14336, 8-bit: gate/up 113 (6.4), down 60 (6.2); sixteen
// tokens, top-8 of 256 and a shared expert, 7168 x 2048, 4-bit: gate/up 255 (6.4), down
// 148 (5.5: a wave has a single unit of a row, and every step of 32 rows a barrier).
// All in one launch, with shares of the steps drawn from counters and waits of the
// workgroups for each other's h and y, took 81 us where these four kernels take 64.
#include <type_traits>

#include "lanes.h"
#include "lds_pipe.h"
#include "split.h"
#include "step.h"

namespace {

using moe::lds::bf16x8;
using moe::lds::u32x4;
using moe::lds::uni;
using moe::lds::uni_ptr;

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kTile = moe::kFewTile;                            // rows of a product
constexpr int kMaxAssign = MOE_FEW_TOKENS * 64;                // k is at most 64
constexpr int kMaxEntries = 256 + kMaxAssign / (kTile + 1) + 1; // experts, and second tiles of those above 16 rows

// Work of a launch. Rows 0 .. N - 1 are the assignments by expert, then token;
// rows N .. N + T - 1 the shared expert's.
struct Few {
    int T, H, E, k, F, SF, N;
    bool two_tiles;                  // entries of up to 32 rows
    int planes;                      // of the router's scores
    int parts, sparts;               // of K in the down projection
    const uint16_t* x;
    const float *logits, *bias;
    const uint8_t *gate, *up, *down, *gate_s, *up_s, *down_s;
    const uint8_t *sgate, *sup, *sdown, *sgate_s, *sup_s, *sdown_s;
    uint16_t *h, *hs;                // [N][F], [T][SF]; the remainders a plane further
    size_t plane;
    float *y, *ys;                   // [parts][N][H], [sparts][T][H]
    int32_t *ids, *err, *row_of;
    float *w, *w_out;
    uint32_t* tables;                // the first kernel's, for the second
    uint16_t* out;
};

// --------------------------------------------------------- router's scores --
// 16 experts against every token over a part of H: each of eight waves takes up to
// kLogitSteps x 32 values of K, their sums meet in LDS, and the parts' are added by
// the choice, in order. (One workgroup an expert on the vector unit took 20 us for
// 16 tokens of 7168; this takes 5.)
constexpr int kLogitSteps = 4;

template <int NT>
__global__ __launch_bounds__(kThreads) void few_logits_kernel(int T, int H, int E, const uint16_t* __restrict__ x,
                                                              const uint16_t* __restrict__ wr, float* __restrict__ logits)
{
    __shared__ f32x4 red[kWaves][NT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
    const int e = min((int)blockIdx.x * kTile + r, E - 1);
    const int k0 = ((int)blockIdx.y * kWaves + wave) * (kLogitSteps * 32) + g * 8;
    const u32x4 none = {0, 0, 0, 0};
    u32x4 a[kLogitSteps], b[NT][kLogitSteps];
#pragma unroll
    for (int i = 0; i < kLogitSteps; ++i) {
        const int k = k0 + i * 32;
        a[i] = k < H ? *reinterpret_cast<const u32x4*>(wr + (size_t)e * H + k) : none;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            b[n][i] = k < H && n * kTile + r < T ? *reinterpret_cast<const u32x4*>(x + (size_t)(n * kTile + r) * H + k) : none;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kLogitSteps; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[i]), __builtin_bit_cast(bf16x8, b[n][i]), acc, 0, 0, 0);
        red[wave][n][lane] = acc;
    }
    __syncthreads();
    // value i of lane l: expert l / 16 * 4 + i, token l % 16
    for (int v = tid; v < NT * 256; v += kThreads) {
        const int n = v / 256, i = v % 256, t = n * kTile + i / 4 % 16, ex = blockIdx.x * kTile + i / 64 * 4 + i % 4;
        float sum = reinterpret_cast<const float*>(red[0][n])[i];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += reinterpret_cast<const float*>(red[w][n])[i];
        if (t < T && ex < E) logits[((size_t)blockIdx.y * T + t) * E + ex] = sum;
    }
}

// -------------------------------------------------------------- the choice --
struct Tables {
    uint8_t tok[kMaxAssign];         // token of a row
    // runs of up to 16 rows of one expert, and the experts with rows (of up to 32)
    int16_t entry_e[kMaxEntries], entry_row[kMaxEntries], live_e[256], live_row[256];
    uint8_t entry_n[kMaxEntries], live_n[256];
    int sums[3][kWaves];
    int entries, live;
};
constexpr int kTableWords = sizeof(Tables) / 4;
static_assert(sizeof(Tables) % 4 == 0 && sizeof(Tables) <= moe::kFewTableBytes, "tables");
struct Choosing {                    // (in the rings' place, before they start)
    uint32_t mask[256];              // tokens that chose the expert
    int16_t base[256];               // its first row
    int16_t id[kMaxAssign];
};

// A score's order as an unsigned integer above 0; NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float s)
{
    const uint32_t b = __float_as_uint(s != s ? -INFINITY : s + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    using namespace moe::lanes;
    v = max(v, (uint32_t)dpp<kQuadXor1>((int)v));
    v = max(v, (uint32_t)dpp<kQuadXor2>((int)v));
    v = max(v, (uint32_t)dpp<kHalfMirror>((int)v));
    v = max(v, (uint32_t)dpp<kMirror>((int)v));
    int lo, hi;
    swap_halves<false>((int)v, lo, hi);
    v = max((uint32_t)lo, (uint32_t)hi);
    swap_halves<true>((int)v, lo, hi);
    return max((uint32_t)lo, (uint32_t)hi);
}

// Top-k of every token (a wave takes tokens wave, wave + 8, ...), then the
// experts' rows and the entries.
__device__ void choose(const Few& f, Tables& s, Choosing& c, bool tell)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    for (int t = wave; t < f.T; t += kWaves) {
        float lg[4];
        uint32_t key[4];
        bool bad = false;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int e = p * 64 + lane;
            lg[p] = 0.0f;
            key[p] = 0;
            if (e < f.E) {
                const float* at = f.logits + (size_t)t * f.E + e;
                float v[moe::kFewLogitParts];
#pragma unroll
                for (int q = 0; q < moe::kFewLogitParts; ++q) v[q] = q < f.planes ? at[(size_t)q * f.T * f.E] : 0.0f;
                float l = v[0];
#pragma unroll
                for (int q = 1; q < moe::kFewLogitParts; ++q) l += v[q];
                const float b = f.bias ? f.bias[e] : 0.0f;
                bad |= !isfinite(l) || !isfinite(b);
                lg[p] = l;
                key[p] = order_of(l + b);
            }
        }
        int my_id = 0;
        float my_lg = -INFINITY;
        for (int j = 0; j < f.k; ++j) {
            const uint32_t m = wave_max(max(max(key[0], key[1]), max(key[2], key[3])));
            int e = 0;
            float l = 0.0f;
#pragma unroll
            for (int p = 3; p >= 0; --p) {  // (the lowest expert of equal scores)
                const uint64_t hit = __ballot(key[p] == m);
                if (hit) {
                    const int at = __builtin_ctzll(hit);
                    e = p * 64 + at;
                    l = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(lg[p]), at));
                }
            }
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (p * 64 + lane == e) key[p] = 0;
            if (lane == j) {
                my_id = e;
                my_lg = l;
            }
        }
        const float top = moe::lanes::group_reduce<64, false>(my_lg);
        const float ex = lane < f.k ? expf(my_lg - top) : 0.0f;
        const float w = ex / moe::lanes::group_reduce<64, true>(ex);
        if (lane < f.k) {
            const int i = t * f.k + lane;
            c.id[i] = (int16_t)my_id;
            if (tell && f.ids) f.ids[i] = my_id;
            if (tell && f.w_out) f.w_out[i] = w;
            if (tell) f.w[i] = w;
        }
        if (tell && __any(bad) && lane == 0) atomicOr(f.err, MOE_ERR_NONFINITE);
    }
    if (tid < 256) c.mask[tid] = 0;
    __syncthreads();
    for (int i = tid; i < f.N; i += kThreads) atomicOr(&c.mask[c.id[i]], 1u << (i / f.k));
    __syncthreads();
    // rows and entries before each expert (threads 0 .. 255 hold one each)
    const int n = tid < 256 ? __popc(c.mask[tid]) : 0, tiles = (n + kTile - 1) / kTile;
    int rows_to = n, tiles_to = tiles, live_to = n > 0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int a = __shfl_up(rows_to, off), b = __shfl_up(tiles_to, off), l = __shfl_up(live_to, off);
        rows_to += lane >= off ? a : 0;
        tiles_to += lane >= off ? b : 0;
        live_to += lane >= off ? l : 0;
    }
    if (lane == 63) {
        s.sums[0][wave] = rows_to;
        s.sums[1][wave] = tiles_to;
        s.sums[2][wave] = live_to;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        rows_to += s.sums[0][w];
        tiles_to += s.sums[1][w];
        live_to += s.sums[2][w];
    }
    if (tid < 256) {
        c.base[tid] = (int16_t)(rows_to - n);
        for (int i = 0; i < tiles; ++i) {
            const int at = tiles_to - tiles + i;
            s.entry_e[at] = (int16_t)tid;
            s.entry_row[at] = (int16_t)(rows_to - n + i * kTile);
            s.entry_n[at] = (uint8_t)min(kTile, n - i * kTile);
        }
        if (n > 0) {
            s.live_e[live_to - 1] = (int16_t)tid;
            s.live_row[live_to - 1] = (int16_t)(rows_to - n);
            s.live_n[live_to - 1] = (uint8_t)n;
        }
    }
    if (tid == kThreads - 1) {
        s.entries = tiles_to;
        s.live = live_to;
    }
    __syncthreads();
    for (int i = tid; i < f.N; i += kThreads) {
        const int t = i / f.k, e = c.id[i];
        const int row = c.base[e] + __popc(c.mask[e] & ((1u << t) - 1u));
        s.tok[row] = (uint8_t)t;
        if (tell) f.row_of[i] = row;
    }
    __syncthreads();
}

// --------------------------------------------------------------- the forms --
// A unit of K: a 128-byte line of 16 weight rows, two times 16 bytes a lane, each
// kSub operands of 32 values (8 a lane). Lane (r, g) = (lane % 16, lane / 16) takes
// row r's chunks of 16 bytes 2 g and 2 g + 1. In LDS a row's chunks are turned so
// that lanes of 16 rows read different banks (see lds_pipe.h). kWords: of four
// scales, of a row's unit. (A unit of 64 bytes of 4-bit codes was slower, whether the
// copies were kept in the caches or not: 307 and 352 us where this takes 257. Chunks g and g + 4 to a
// lane, which bring fewer conflicts in the LDS, took the same time.)
template <int FORM>
struct Form;
template <>
struct Form<MOE_W_BF16> {
    static constexpr int kUnit = 64, kSub = 1, kWords = 0;
    __device__ static size_t bytes(size_t n) { return 2 * n; }
};
template <>
struct Form<MOE_W_MX8> {
    static constexpr int kUnit = 128, kSub = 2, kWords = 1;
    __device__ static size_t bytes(size_t n) { return n; }
};
template <>
struct Form<MOE_W_MX4> {
    static constexpr int kUnit = 256, kSub = 4, kWords = 2;
    __device__ static size_t bytes(size_t n) { return n / 2; }
};

constexpr int kUnitBytes = 128, kLoads = 2;

// One load's operands. s: the scale of its block of 32 values.
template <int FORM>
__device__ __forceinline__ void widen(const u32x4& c, float s, bf16x8 (&o)[Form<FORM>::kSub])
{
    if constexpr (FORM == MOE_W_BF16) {
        o[0] = __builtin_bit_cast(bf16x8, c);
    } else {
#pragma unroll
        for (int j = 0; j < Form<FORM>::kSub; ++j) {
            u32x4 w;
            if constexpr (FORM == MOE_W_MX8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * j + i], s, false));
                    w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * j + i], s, true));
                }
            } else {
                w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], s, 0));
                w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], s, 1));
                w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], s, 2));
                w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], s, 3));
            }
            o[j] = __builtin_bit_cast(bf16x8, w);
        }
    }
}

// A wave's ring of weights: items are units of one stream, in the order unit, then
// stream; kItems of them in flight, each two copies of 8 rows (1 KB). The scales of
// a step's units come in copies of four words a row ahead of its first item, into a
// ring of steps of their own.
template <int FORM, int NU>
struct Ring {
    static constexpr int kWords = NU * Form<FORM>::kWords;
    static constexpr int kPerStep = 2 * NU, kCopies = 2, kItems = kWords ? 6 : 7;
    static constexpr int kScaleCopies = 2 * ((kWords + 3) / 4);             // of a step
    static constexpr int kSteps = (kItems + kPerStep - 1) / kPerStep + 1;   // whose scales are in flight or in use
    static constexpr int kItem = kCopies * 1024, kScales = kItems * kItem, kBytes = kScales + kSteps * kScaleCopies * 256;
    // Copies that may still be out when items up to `landed` of a step have to be
    // there, items up to `issued` having been started.
    static constexpr int out(int landed, int issued)
    {
        return (issued - landed) * kCopies + (issued / kPerStep - landed / kPerStep) * kScaleCopies;
    }
};
constexpr int kRingBytes = 14 * 1024;  // a wave's, the most of all rings

// Waits until at most VM of the wave's memory operations are out, and for its LDS
// reads.
template <int VM>
__device__ __forceinline__ void landed()
{
    static_assert(VM >= 0 && VM < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(VM) : "memory");
}

// f(0), f(1), ... with the number as a constant.
template <typename F, int... J>
__device__ __forceinline__ void unrolled(F f, std::integer_sequence<int, J...>)
{
    (f(std::integral_constant<int, J>{}), ...);
}

// The waves' sums of one step, [wave][stream][lane], doubled (for two steps in turn, or
// the two tiles of a step).
struct Reduce {
    f32x4 v[2][kWaves][2][64];
};

// Steps s0 .. s1 of one entry. w, sc: the two streams' weights and scales at the
// entry's first weight row (stream 1: up, or 16 rows on), `rows` of them, of K
// values; step_rows weight rows from a step to the next; u0, cnt: this
// wave's units of K. load(b) fetches the rows' values of those units (NB 2: and
// their remainders; TB 2: of both tiles of 16 rows). ring: the wave's LDS. done(step,
// sums of both streams, tile) is called by 256 threads of a tile: thread e has weight
// row e / 64 % 4 * 4 + e % 4 of the step's and the tile's row e / 4 % 16.
template <int FORM, int NU, int TB, int NB, typename Load, typename Done>
__device__ __forceinline__ void run_steps(const uint8_t* const (&w)[2], const uint8_t* const (&sc)[2], int K, int rows, int step_rows,
                                          int u0, int cnt, int s0, int s1, const char* ring, Load load, Reduce& red,
                                          int& turn, Done done)
{
    using FM = Form<FORM>;
    using RG = Ring<FORM, NU>;
    static_assert(RG::kBytes <= kRingBytes, "ring");
    constexpr int I = RG::kPerStep, D = RG::kItems;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = (uint32_t)FM::bytes(K), step_bytes = (uint32_t)step_rows * row_bytes, bytes = (uint32_t)rows * row_bytes;
    const uint32_t srow = (uint32_t)(K / 32), sstep = (uint32_t)step_rows * srow, sbytes = (uint32_t)rows * srow;
    const uint32_t ring_u = (uint32_t)(uintptr_t)ring;
    // this lane's 16 bytes of a copy of 8 rows (a second copy's rows are 8 on, their
    // chunks four places further round), and where it reads its operands
    const int cr = lane >> 3, cc = (lane & 7) ^ moe::lds::swz(cr);
    const uint32_t first = (uint32_t)cr * row_bytes + (uint32_t)u0 * kUnitBytes;
    const uint32_t voff[2] = {first + 16u * cc, first + 16u * (cc ^ 4)};
    const uint32_t svoff = (uint32_t)(lane >> 2) * srow + 4u * (u0 * FM::kWords + (lane & 3));
    const uint32_t from[2] = {(uint32_t)(r * 128 + ((2 * g) ^ moe::lds::swz(r)) * 16),
                              (uint32_t)(r * 128 + ((2 * g + 1) ^ moe::lds::swz(r)) * 16)};

    int to = 0, sto = 0, sat = 0;  // ring places: the next item's copies, scales' copies, scales' reads
    auto issue = [&](int s, int j) {  // item j of step s
        const int u = j / 2, m = j % 2;
        if (RG::kWords && j == 0) {
#pragma unroll
            for (int i = 0; i < RG::kScaleCopies; ++i)
                moe::lds::copy4(moe::lds::buffer_of(sc[i % 2], s < s1 ? sbytes : 0u), svoff, (int)((uint32_t)s * sstep + i / 2 * 16),
                                ring_u + RG::kScales + (sto * RG::kScaleCopies + i) * 256);
            sto = sto + 1 == RG::kSteps ? 0 : sto + 1;
        }
#pragma unroll
        for (int i = 0; i < RG::kCopies; ++i)
            moe::lds::copy16<true>(moe::lds::buffer_of(w[m], s < s1 && u < cnt ? bytes : 0u), voff[i],
                                   (int)((uint32_t)s * step_bytes + u * kUnitBytes + i * 8 * row_bytes), ring_u + to + i * 1024);
        to = to + RG::kItem == RG::kScales ? 0 : to + RG::kItem;
    };
    u32x4 next[kLoads];
    uint32_t words[2][RG::kWords ? RG::kWords : 1];
    int at = 0;  // ring place of the next item to read
    auto read = [&]() {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) next[i] = *reinterpret_cast<const u32x4*>(ring + at + from[i]);
        at = at + RG::kItem == RG::kScales ? 0 : at + RG::kItem;
    };
    auto read_scales = [&]() {
        if constexpr (RG::kWords > 0) {
            const char* p = ring + RG::kScales + sat * RG::kScaleCopies * 256 + r * 16;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < RG::kWords; ++i) words[m][i] = *reinterpret_cast<const uint32_t*>(p + (i / 4 * 2 + m) * 256 + i % 4 * 4);
            sat = sat + 1 == RG::kSteps ? 0 : sat + 1;
        }
    };
    // The scale of load i of unit u of stream m, in this lane. (Past this wave's units
    // and past K the words are others', maybe NaN, on values of 0: half of the last
    // unit of 256 values can be.)
    auto scale = [&](int m, int u, int i) {
        if constexpr (RG::kWords == 0) return 0.0f;
        const bool in = u < cnt && (FM::kWords == 1 || (u0 + u) * FM::kUnit + g * (FM::kUnit / 4) < K);
        const uint32_t word = FM::kWords == 1 ? words[m][u] : g < 2 ? words[m][2 * u] : words[m][2 * u + 1];
        const uint32_t byte = word >> (FM::kWords == 1 ? 8 * g : 16 * (g & 1) + 8 * i);
        return __uint_as_float(in ? (byte & 255u) << 23 : 0u);
    };
#pragma unroll
    for (int j = 0; j < D; ++j) issue(s0 + j / I, j % I);
    bf16x8 b[TB][NB][NU * kLoads * FM::kSub];
    load(b);
    landed<0>();
    read();
    read_scales();
    for (int s = s0; s < s1; ++s) {
        f32x4 acc[TB][2];
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[t][0] = acc[t][1] = f32x4{0, 0, 0, 0};
        float f[2][NU][FM::kWords == 2 ? 2 : 1];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < (FM::kWords == 2 ? 2 : 1); ++i) f[m][u][i] = scale(m, u, i);
        unrolled([&](auto j_tag) {
            constexpr int j = decltype(j_tag)::value, u = j / 2, m = j % 2;
            // the next item is there; this one is in registers and its place free
            landed<RG::out(j + 1, j + D - 1)>();
            u32x4 c[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) c[i] = next[i];
            issue(s + (j + D) / I, (j + D) % I);
            read();
            if (j + 1 == I) read_scales();
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                bf16x8 a[FM::kSub];
                widen<FORM>(c[i], f[m][u][FM::kWords == 2 ? i : 0], a);
#pragma unroll
                for (int q = 0; q < FM::kSub; ++q)
#pragma unroll
                    for (int t = 0; t < TB; ++t)
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            acc[t][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q], b[t][n][(u * kLoads + i) * FM::kSub + q], acc[t][m], 0, 0, 0);
            }
        }, std::make_integer_sequence<int, I>{});
        if (TB == 2) moe::lds::slot_barrier();  // (the step before's sums have been read)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int m = 0; m < 2; ++m) red.v[TB == 2 ? t : turn][wave][m][lane] = acc[t][m];
        moe::lds::wait_vm_lgkm<63>();  // the sums are in LDS; copies stay in flight
        moe::lds::slot_barrier();
        // one half of the waves adds them up, the other goes on, in turns (or each half
        // a tile): a value of each stream a thread, in the waves' order
        if (TB == 2 || (wave >> 2) == (s & 1)) {
            const int e = threadIdx.x & 255, from = TB == 2 ? wave >> 2 : turn;
            float x[kWaves], y[kWaves];
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                x[v] = reinterpret_cast<const float*>(red.v[from][v][0])[e];
                y[v] = reinterpret_cast<const float*>(red.v[from][v][1])[e];
            }
#pragma unroll
            for (int v = 1; v < kWaves; ++v) {
                x[0] += x[v];
                y[0] += y[v];
            }
            done(s, x[0], y[0], TB == 2 ? wave >> 2 : 0);
        }
        turn ^= 1;
    }
    landed<0>();  // copies of nothing past the last step
    if (TB == 2) moe::lds::slot_barrier();  // (the next entry's sums may have one tile: no barrier before they are written)
}

// Values of an entry's rows as operands: lane (n, g) takes of row n, at `row`, of
// width K, what lane (r, g) takes of a weight row in units u0 .. u0 + cnt.
template <int FORM, int NU, int N>
__device__ __forceinline__ void load_rows(const uint16_t* row, bool in, int K, int u0, int cnt, bf16x8 (&b)[N])
{
    using FM = Form<FORM>;
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int j = 0; j < FM::kSub; ++j) {
                const int at = (u0 + u) * FM::kUnit + ((g * kLoads + i) * FM::kSub + j) * 8;
                u32x4 v = {0, 0, 0, 0};
                if (in && u < cnt && at < K) v = *reinterpret_cast<const u32x4*>(row + at);
                b[(u * kLoads + i) * FM::kSub + j] = __builtin_bit_cast(bf16x8, v);
            }
}

// This workgroup's run of `total` steps.
__device__ __forceinline__ void my_run(int64_t total, int& a, int& z)
{
    a = uni((int)(total * blockIdx.x / gridDim.x));
    z = uni((int)(total * (blockIdx.x + 1) / gridDim.x));
}

// ---------------------------------------------------------------- gate, up --
// a and b as two bf16 each: their rounding, a pair a word, and what it leaves of them (lo).
// A value that would round to an infinity is cut, so that what is left is finite; an
// infinite one leaves nothing. (As a difference either would be infinite or NaN, and out NaN.)
__device__ __forceinline__ uint32_t two_bf16(float a, float b, uint32_t& lo)
{
    uint32_t hi = moe::pack_bf16x2(a, b);
    if ((hi & 0x7fffu) == 0x7f80u) hi = (hi & 0xffff0000u) | __float_as_uint(a) >> 16;
    if ((hi & 0x7fff0000u) == 0x7f800000u) hi = (hi & 0xffffu) | (__float_as_uint(b) & 0xffff0000u);
    const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xffff0000u);
    lo = moe::pack_bf16x2(isinf(a) ? 0.0f : ra, isinf(b) ? 0.0f : rb);
    return hi;
}

// TB: tiles of 16 rows that an entry has at most.
template <int FORM, int NU, int TB>
__global__ __launch_bounds__(kThreads, 2) void few_gateup_kernel(const Few f)
{
    using FM = Form<FORM>;
    __shared__ Tables tab;
    __shared__ Reduce red;
    __shared__ __attribute__((aligned(1024))) char rings[kWaves * kRingBytes];
    choose(f, tab, *reinterpret_cast<Choosing*>(rings), blockIdx.x == 0);
    if (blockIdx.x == 0)   // (the next kernel reads them: 19 us for one token on bf16 weights, 22 where it chooses again)
        for (int i = threadIdx.x; i < kTableWords; i += kThreads) f.tables[i] = reinterpret_cast<const uint32_t*>(&tab)[i];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), n = lane & 15;
    const int en = threadIdx.x / 4 % 16, ew = threadIdx.x / 64 % 4 * 4 + threadIdx.x % 4;  // run_steps' done: row, column
    const int per = f.F / kTile, sper = f.SF / kTile, entries = uni(TB == 2 ? tab.live : tab.entries), sentries = f.SF ? (f.T + TB * kTile - 1) / (TB * kTile) : 0;
    const int units = (f.H + FM::kUnit - 1) / FM::kUnit, u0 = uni(wave * units / kWaves), cnt = uni((wave + 1) * units / kWaves) - u0;
    const char* ring = rings + wave * kRingBytes;
    int at, end, turn = 0;
    my_run((int64_t)entries * per + (int64_t)sentries * sper, at, end);
    while (at < end) {
        const bool shared = at >= entries * per;
        const int local = shared ? at - entries * per : at, each = shared ? sper : per;
        const int entry = uni(local / each), s0 = local - entry * each, s1 = min(each, s0 + end - at);
        const int e = shared ? 0 : uni((int)(TB == 2 ? tab.live_e : tab.entry_e)[entry]);
        const int row0 = shared ? entry * TB * kTile : uni((int)(TB == 2 ? tab.live_row : tab.entry_row)[entry]);
        const int rows = shared ? min(TB * kTile, f.T - row0) : uni((int)(TB == 2 ? tab.live_n : tab.entry_n)[entry]);
        const size_t first = (size_t)e * f.F;
        const uint8_t* const w[2] = {(shared ? f.sgate : f.gate) + FM::bytes(first * f.H),
                                     (shared ? f.sup : f.up) + FM::bytes(first * f.H)};
        const uint8_t* const sc[2] = {(shared ? f.sgate_s : f.gate_s) + first * (f.H / 32),
                                      (shared ? f.sup_s : f.up_s) + first * (f.H / 32)};
        auto load = [&](auto& b) {
#pragma unroll
            for (int t = 0; t < (int)(sizeof(b) / sizeof(b[0])); ++t) {
                const int r = t * kTile + n, tok = r < rows ? (shared ? row0 + r : (int)tab.tok[row0 + r]) : 0;
                load_rows<FORM, NU>(f.x + (size_t)tok * f.H, r < rows, f.H, u0, cnt, b[t][0]);
            }
        };
        const int width = shared ? f.SF : f.F;
        uint16_t* h = (shared ? f.hs : f.h) + (size_t)(row0 + en) * width + ew;
        auto done = [&](int s, float g, float u, int t) {
            // (an even thread stores its neighbour's column too)
            const float v = moe::silu(g) * u, v1 = moe::lanes::dpp<moe::lanes::kQuadXor1>(v);
            uint32_t lo;
            const uint32_t hi = two_bf16(v, v1, lo);
            if (t * kTile + en < rows && threadIdx.x % 2 == 0) {
                uint16_t* to = h + (size_t)(t * kTile) * width + s * kTile;
                *reinterpret_cast<uint32_t*>(to) = hi;
                *reinterpret_cast<uint32_t*>(to + f.plane) = lo;
            }
        };
        if (TB == 1 || rows <= kTile) run_steps<FORM, NU, 1, 1>(w, sc, f.H, width, kTile, u0, cnt, s0, s1, ring, load, red, turn, done);
        else run_steps<FORM, NU, TB, 1>(w, sc, f.H, width, kTile, u0, cnt, s0, s1, ring, load, red, turn, done);
        at += s1 - s0;
    }
}

// -------------------------------------------------------------------- down --
template <int FORM, int NU, int TB>
__global__ __launch_bounds__(kThreads, 2) void few_down_kernel(const Few f)
{
    using FM = Form<FORM>;
    __shared__ Tables tab;
    __shared__ Reduce red;
    __shared__ __attribute__((aligned(1024))) char rings[kWaves * kRingBytes];
    for (int i = threadIdx.x; i < kTableWords; i += kThreads) reinterpret_cast<uint32_t*>(&tab)[i] = f.tables[i];
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), n = lane & 15;
    const int en = threadIdx.x / 4 % 16, ew = threadIdx.x / 64 % 4 * 4 + threadIdx.x % 4;  // run_steps' done: row, column
    const int entries = uni(TB == 2 ? tab.live : tab.entries), sentries = f.SF ? (f.T + TB * kTile - 1) / (TB * kTile) : 0, each = f.H / (2 * kTile);
    const char* ring = rings + wave * kRingBytes;
    int at, end, turn = 0;
    my_run((int64_t)each * (entries * f.parts + sentries * f.sparts), at, end);
    while (at < end) {
        int item = uni(at / each);
        const int s0 = at - item * each, s1 = min(each, s0 + end - at);
        const bool shared = item >= entries * f.parts;
        if (shared) item -= entries * f.parts;
        const int parts = shared ? f.sparts : f.parts, entry = uni(item / parts), part = item - entry * parts;
        const int e = shared ? 0 : uni((int)(TB == 2 ? tab.live_e : tab.entry_e)[entry]);
        const int row0 = shared ? entry * TB * kTile : uni((int)(TB == 2 ? tab.live_row : tab.entry_row)[entry]);
        const int rows = shared ? min(TB * kTile, f.T - row0) : uni((int)(TB == 2 ? tab.live_n : tab.entry_n)[entry]);
        const int K = shared ? f.SF : f.F, units = (K + FM::kUnit - 1) / FM::kUnit;
        const int p0 = uni(moe::part_begin(part, units, parts)), pn = uni(moe::part_begin(part + 1, units, parts)) - p0;
        const int u0 = p0 + uni(wave * pn / kWaves), cnt = p0 + uni((wave + 1) * pn / kWaves) - u0;
        const size_t first = (size_t)e * f.H;
        const uint8_t* base = (shared ? f.sdown : f.down) + FM::bytes(first * K);
        const uint8_t* sbase = (shared ? f.sdown_s : f.down_s) + first * (K / 32);
        const uint8_t* const w[2] = {base, base + FM::bytes((size_t)kTile * K)};
        const uint8_t* const sc[2] = {sbase, sbase + kTile * (K / 32)};
        auto load = [&](auto& b) {
#pragma unroll
            for (int t = 0; t < (int)(sizeof(b) / sizeof(b[0])); ++t) {
                const bool in = t * kTile + n < rows;
                const uint16_t* h = (shared ? f.hs : f.h) + (size_t)(row0 + (in ? t * kTile + n : 0)) * K;
                load_rows<FORM, NU>(h, in, K, u0, cnt, b[t][0]);
                load_rows<FORM, NU>(h + f.plane, in, K, u0, cnt, b[t][1]);
            }
        };
        float* y = (shared ? f.ys + (size_t)part * f.T * f.H : f.y + (size_t)part * f.N * f.H) +
                   (size_t)(row0 + en) * f.H + ew;
        auto done = [&](int s, float a, float c, int t) {
            if (t * kTile + en < rows) {
                float* to = y + (size_t)(t * kTile) * f.H + s * 2 * kTile;
                to[0] = a;
                to[kTile] = c;
            }
        };
        if (TB == 1 || rows <= kTile) run_steps<FORM, NU, 1, 2>(w, sc, K, f.H - kTile, 2 * kTile, u0, cnt, s0, s1, ring, load, red, turn, done);
        else run_steps<FORM, NU, TB, 2>(w, sc, K, f.H - kTile, 2 * kTile, u0, cnt, s0, s1, ring, load, red, turn, done);
        at += s1 - s0;
    }
}

// ----------------------------------------------------------------- combine --
__global__ __launch_bounds__(256) void few_combine_kernel(const Few f)
{
    const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= f.H) return;
    f32x4 sum = {0, 0, 0, 0};
    for (int j = 0; j < f.k; ++j) {
        const int i = t * f.k + j, row = f.row_of[i];
        f32x4 v = *reinterpret_cast<const f32x4*>(f.y + (size_t)row * f.H + c);
        for (int p = 1; p < f.parts; ++p) v += *reinterpret_cast<const f32x4*>(f.y + ((size_t)p * f.N + row) * f.H + c);
        const float w = f.w[i];
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[q] = fmaf(w, v[q], sum[q]);
    }
    for (int p = 0; p < f.sparts; ++p) sum += *reinterpret_cast<const f32x4*>(f.ys + ((size_t)p * f.T + t) * f.H + c);
    *reinterpret_cast<uint2*>(f.out + (size_t)t * f.H + c) =
        make_uint2(moe::pack_bf16x2(sum[0], sum[1]), moe::pack_bf16x2(sum[2], sum[3]));
}

// ----------------------------------------------------------------- launches --

int cu_count()
{
    static const int cus = [] {
        int dev = 0, n = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
            n = moe::kGemmMaxGrid;
        return n;
    }();
    return cus;
}

hipError_t launch_logits(const moe_shape_t& s, const MoeFew& a, float* logits, hipStream_t st)
{
    static_assert(moe::kFewLogitK == kWaves * kLogitSteps * 32, "a workgroup's part of H");
    const uint16_t *x = static_cast<const uint16_t*>(a.x), *w = static_cast<const uint16_t*>(a.w_router);
    const dim3 grid((s.E + kTile - 1) / kTile, moe::few_logit_parts(s.H));
    if (s.T <= kTile) few_logits_kernel<1><<<grid, kThreads, 0, st>>>(s.T, s.H, s.E, x, w, logits);
    else few_logits_kernel<2><<<grid, kThreads, 0, st>>>(s.T, s.H, s.E, x, w, logits);
    return hipGetLastError();
}

// Units of K that a wave takes at most, as the kernels' NU: 8192 values of H (4096 where
// an entry has two tiles, whose rows take twice the registers), 4096 or 2048 of a part
// of F. Of a wider x gate/up takes entries of 16 rows, and an expert with more reads
// those weights twice. (14 units of bf16 and 7 of 8-bit codes, for an x of 7168, against
// 16 and 8, top-8 of experts of 2048, us: bf16, 1 and 8 of 256 experts' tokens, 126.4 and
// 126.6, 805 and 805; 8-bit, 1 token 86.4 and 87.2, 16 of 64 experts 474 and 480.)
template <int FORM, int TB>
hipError_t launch_gateup(const Few& f, int grid, hipStream_t st)
{
    const int units = (f.H + Form<FORM>::kUnit - 1) / Form<FORM>::kUnit, n = (units + kWaves - 1) / kWaves;
#define MOE_FEW(N) few_gateup_kernel<FORM, N, TB><<<grid, kThreads, 0, st>>>(f)
    if constexpr (FORM == MOE_W_BF16) {
        if (n <= 2) MOE_FEW(2);
        else if (n <= 4) MOE_FEW(4);
        else if (n <= 8) MOE_FEW(8);
        if constexpr (TB == 1) {
            if (n > 14) MOE_FEW(16);
            else if (n > 8) MOE_FEW(14);
        }
    } else if constexpr (FORM == MOE_W_MX8) {
        if (n <= 1) MOE_FEW(1);
        else if (n <= 2) MOE_FEW(2);
        else if (n <= 4) MOE_FEW(4);
        if constexpr (TB == 1) {
            if (n > 7) MOE_FEW(8);
            else if (n > 4) MOE_FEW(7);
        }
    } else {
        if (n <= 1) MOE_FEW(1);
        else if (n <= 2) MOE_FEW(2);
        if constexpr (TB == 1)
            if (n > 2) MOE_FEW(4);
    }
#undef MOE_FEW
    return hipGetLastError();
}

template <int FORM, int TB>
hipError_t launch_down(const Few& f, int grid, hipStream_t st)
{
    auto most = [&](int K, int parts) {
        const int units = (K + Form<FORM>::kUnit - 1) / Form<FORM>::kUnit, part = parts ? (units + parts - 1) / parts : 0;
        return (part + kWaves - 1) / kWaves;
    };
    const int n = most(f.F, f.parts) > most(f.SF, f.sparts) ? most(f.F, f.parts) : most(f.SF, f.sparts);
#define MOE_FEW(N) few_down_kernel<FORM, N, TB><<<grid, kThreads, 0, st>>>(f)
    constexpr int kMost = moe::kFewPart / TB / Form<FORM>::kUnit / kWaves;  // 8, 4, 2 or, of two tiles, 4, 2, 1
    if constexpr (kMost >= 8) {
        if (n <= 2) MOE_FEW(2);
        else if (n <= 4) MOE_FEW(4);
        else MOE_FEW(8);
    } else if constexpr (kMost >= 4) {
        if (n <= kMost / 4) MOE_FEW(kMost / 4);
        else if (n <= kMost / 2) MOE_FEW(kMost / 2);
        else MOE_FEW(kMost);
    } else if constexpr (kMost == 2) {
        if (n <= 1) MOE_FEW(1);
        else MOE_FEW(2);
    } else {
        MOE_FEW(1);
    }
#undef MOE_FEW
    return hipGetLastError();
}

template <int FORM>
hipError_t launch_form(const Few& f, hipStream_t st)
{
    const int grid = cu_count();
    const bool two = f.two_tiles;
    const hipError_t e = two && f.H <= moe::kFewMaxH / 2 ? launch_gateup<FORM, 2>(f, grid, st) : launch_gateup<FORM, 1>(f, grid, st);
    if (e != hipSuccess) return e;
    return two ? launch_down<FORM, 2>(f, grid, st) : launch_down<FORM, 1>(f, grid, st);
}

}  // namespace

hipError_t moe_launch_few(const moe_shape_t& s, const MoeFew& a, char* ws, hipStream_t st)
{
    if (s.T == 0) return hipSuccess;
    const moe::FewWsLayout L = moe::few_ws_layout(s, a.shared_F);
    auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
    Few f;
    f.T = s.T, f.H = s.H, f.E = s.E, f.k = s.k, f.F = s.F, f.SF = a.shared_F, f.N = s.T * s.k;
    f.planes = moe::few_logit_parts(s.H);
    f.two_tiles = moe::few_two_tiles(s);
    f.parts = moe::few_parts(s.F, f.two_tiles), f.sparts = moe::few_parts(a.shared_F, f.two_tiles);
    f.x = static_cast<const uint16_t*>(a.x);
    float* logits = reinterpret_cast<float*>(ws + L.logits);
    f.logits = logits, f.bias = a.bias;
    f.gate = u8(a.routed.gate), f.up = u8(a.routed.up), f.down = u8(a.routed.down);
    f.gate_s = u8(a.routed.gate_scales), f.up_s = u8(a.routed.up_scales), f.down_s = u8(a.routed.down_scales);
    f.sgate = u8(a.shared.gate), f.sup = u8(a.shared.up), f.sdown = u8(a.shared.down);
    f.sgate_s = u8(a.shared.gate_scales), f.sup_s = u8(a.shared.up_scales), f.sdown_s = u8(a.shared.down_scales);
    f.h = reinterpret_cast<uint16_t*>(ws + L.h), f.hs = f.h + L.h_shared, f.plane = L.h_plane;
    f.y = reinterpret_cast<float*>(ws + L.y), f.ys = f.y + L.y_shared;
    f.ids = a.ids, f.err = a.err, f.row_of = reinterpret_cast<int32_t*>(ws + L.row_of);
    f.w = reinterpret_cast<float*>(ws + L.w), f.w_out = a.w;
    f.tables = reinterpret_cast<uint32_t*>(ws + L.tables);
    f.out = static_cast<uint16_t*>(a.out);
    hipError_t e = launch_logits(s, a, logits, st);
    if (e != hipSuccess) return e;
    e = a.form == MOE_W_BF16 ? launch_form<MOE_W_BF16>(f, st)
        : a.form == MOE_W_MX8 ? launch_form<MOE_W_MX8>(f, st) : launch_form<MOE_W_MX4>(f, st);
    if (e != hipSuccess) return e;
    few_combine_kernel<<<dim3((s.H + 1023) / 1024, s.T), 256, 0, st>>>(f);
    return hipGetLastError();
}
