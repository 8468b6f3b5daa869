// few.hip -- a whole MoE layer for up to 32 tokens (moe_few_layer).
//
//   logits = x Wr^T; top-k of logits + bias; w = softmax of the chosen logits;
//   out = sum_j w_j Wd (silu(Wg x) * (Wu x)) (+ the shared expert).
//
// Bound by the live experts' weights, each read once. A step is 16 weight rows
// of two streams (gate and up; in the down projection, two neighbours) times up
// to 16 rows of one expert: the weights go from memory into the registers as
// operands of v_mfma_f32_16x16x32_bf16 (codes are widened to bf16, exactly), the
// rows' values stay in registers from step to step. The eight waves of a
// workgroup share K; their sums meet in LDS. A workgroup takes a run of
// neighbouring steps, so that it changes its expert rarely, and holds up to 16
// loads of 16 bytes a lane in flight across steps.
//
// h = silu(g) u is kept as two bf16 (value and remainder), so that it carries 16
// bits into the down projection; its sums are kept in fp32 for each assignment
// and added in j order.
#include <type_traits>

#include "lanes.h"
#include "lds_pipe.h"
#include "step.h"

namespace {

using moe::lds::bf16x8;
using moe::lds::u32x4;
using moe::lds::uni;
using moe::lds::uni_ptr;

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kTile = 16;                                      // rows of an entry
constexpr int kMaxAssign = MOE_FEW_TOKENS * 64;                // k is at most 64
constexpr int kMaxEntries = 256 + kMaxAssign / (kTile + 1) + 1; // experts, and second tiles of those above 16 rows

// Work of a launch. Rows 0 .. N - 1 are the assignments by expert, then token;
// rows N .. N + T - 1 the shared expert's.
struct Few {
    int T, H, E, k, F, SF, N;
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
    uint16_t* out;
};

// --------------------------------------------------------- router's scores --
// One workgroup an expert: its row against every token's, fp32 sums in an order
// fixed by H.
template <int TT>
__global__ __launch_bounds__(256) void few_logits_kernel(int T, int H, int E, const uint16_t* __restrict__ x,
                                                         const uint16_t* __restrict__ wr, float* __restrict__ logits)
{
    __shared__ float red[4][TT];
    const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.0f;
    for (int c = tid * 8; c < H; c += 256 * 8) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(wr + (size_t)e * H + c);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(x + (size_t)(t < T ? t : 0) * H + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[t] = fmaf(__uint_as_float(w[i] << 16), __uint_as_float(v[i] << 16), acc[t]);
                acc[t] = fmaf(__uint_as_float(w[i] & 0xffff0000u), __uint_as_float(v[i] & 0xffff0000u), acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const float s = moe::lanes::group_reduce<64, true>(acc[t]);
        if (lane == 0) red[wave][t] = s;
    }
    __syncthreads();
    if (tid < T) logits[(size_t)tid * E + e] = red[0][tid] + red[1][tid] + red[2][tid] + red[3][tid];
}

// -------------------------------------------------------------- the choice --
struct Tables {
    uint32_t mask[256];              // tokens that chose the expert
    int16_t base[256];               // its first row
    int16_t id[kMaxAssign], row_of[kMaxAssign];
    float w[kMaxAssign];
    uint8_t tok[kMaxAssign];         // token of a row
    int16_t entry_e[kMaxEntries], entry_row[kMaxEntries];
    uint8_t entry_n[kMaxEntries];
    int sums[2][kWaves];
    int entries;                     // of routed experts
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
// experts' rows and the entries: runs of up to 16 rows of one expert.
__device__ void choose(const Few& f, Tables& s, bool tell)
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
                const float l = f.logits[(size_t)t * f.E + e], b = f.bias ? f.bias[e] : 0.0f;
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
            s.id[i] = (int16_t)my_id;
            s.w[i] = w;
            if (tell && f.ids) f.ids[i] = my_id;
            if (tell && f.w_out) f.w_out[i] = w;
            if (tell) f.w[i] = w;
        }
        if (tell && __any(bad) && lane == 0) atomicOr(f.err, MOE_ERR_NONFINITE);
    }
    if (tid < 256) s.mask[tid] = 0;
    __syncthreads();
    for (int i = tid; i < f.N; i += kThreads) atomicOr(&s.mask[s.id[i]], 1u << (i / f.k));
    __syncthreads();
    // rows and entries before each expert (threads 0 .. 255 hold one each)
    const int n = tid < 256 ? __popc(s.mask[tid]) : 0, tiles = (n + kTile - 1) / kTile;
    int rows_to = n, tiles_to = tiles;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int a = __shfl_up(rows_to, off), b = __shfl_up(tiles_to, off);
        rows_to += lane >= off ? a : 0;
        tiles_to += lane >= off ? b : 0;
    }
    if (lane == 63) {
        s.sums[0][wave] = rows_to;
        s.sums[1][wave] = tiles_to;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        rows_to += s.sums[0][w];
        tiles_to += s.sums[1][w];
    }
    if (tid < 256) {
        s.base[tid] = (int16_t)(rows_to - n);
        for (int i = 0; i < tiles; ++i) {
            const int at = tiles_to - tiles + i;
            s.entry_e[at] = (int16_t)tid;
            s.entry_row[at] = (int16_t)(rows_to - n + i * kTile);
            s.entry_n[at] = (uint8_t)min(kTile, n - i * kTile);
        }
    }
    if (tid == kThreads - 1) s.entries = tiles_to;
    __syncthreads();
    for (int i = tid; i < f.N; i += kThreads) {
        const int t = i / f.k, e = s.id[i];
        const int row = s.base[e] + __popc(s.mask[e] & ((1u << t) - 1u));
        s.row_of[i] = (int16_t)row;
        s.tok[row] = (uint8_t)t;
        if (tell) f.row_of[i] = row;
    }
    __syncthreads();
}

// --------------------------------------------------------------- the forms --
// A unit of K: kLoads loads of 16 bytes a lane, each kSub operands of 32 values
// (8 a lane). Lane (r, g) = (lane % 16, lane / 16) holds row r, and of the unit the
// values of bytes (g * kLoads + q) * 16 on in load q: both loads of a 128-byte unit
// touch the whole line.
template <int FORM>
struct Form;
template <>
struct Form<MOE_W_BF16> {
    static constexpr int kUnit = 64, kLoads = 2, kSub = 1, kUnitBytes = 128;
    __device__ static size_t bytes(size_t n) { return 2 * n; }
};
template <>
struct Form<MOE_W_MX8> {
    static constexpr int kUnit = 128, kLoads = 2, kSub = 2, kUnitBytes = 128;
    __device__ static size_t bytes(size_t n) { return n; }
};
template <>
struct Form<MOE_W_MX4> {
    static constexpr int kUnit = 128, kLoads = 1, kSub = 4, kUnitBytes = 64;
    __device__ static size_t bytes(size_t n) { return n / 2; }
};

// One load's operands. scales: the row's four scale bytes of the unit.
template <int FORM>
__device__ __forceinline__ void widen(const u32x4& c, uint32_t scales, int g, bf16x8 (&o)[Form<FORM>::kSub])
{
    if constexpr (FORM == MOE_W_BF16) {
        o[0] = __builtin_bit_cast(bf16x8, c);
    } else {
        const uint32_t byte = (scales >> (8 * g)) & 255u;
        const float s = __uint_as_float(byte << 23);
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

// Loads in flight across steps: 16, or 14 where a step's are a multiple of 7 (8 where
// the rows' values fill the registers).
constexpr int ring_of(int loads) { return loads % 7 == 0 ? 14 : loads == 64 ? 8 : 16; }

// 16 bytes a lane through a buffer of `records` bytes, not kept in the caches. A
// load past them reads nothing and gives zeros, each of its four words by itself
// (the hardware's check of a buffer's range), so a load of nothing has records 0.
__device__ __forceinline__ u32x4 load16(const uint8_t* base, uint32_t records, uint32_t voff, uint32_t soff)
{
    const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, (int)records, 0x00020000);
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 2));
}

// N words (1, 2, 3 or 4) a lane, kept in the caches. No more than are used: a word of
// a load in flight that nobody reads is a free register to the compiler, which then
// waits for every load before it takes it.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* base, uint32_t records, uint32_t voff, uint32_t soff, uint32_t* w)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
    const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, (int)records, 0x00020000);
    if constexpr (N == 1) {
        w[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)voff, (int)soff, 0);
    } else if constexpr (N == 2) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)voff, (int)soff, 0));
        w[0] = v[0], w[1] = v[1];
    } else if constexpr (N == 3) {
        const u32x3 v = __builtin_bit_cast(u32x3, __builtin_amdgcn_raw_buffer_load_b96(r, (int)voff, (int)soff, 0));
        w[0] = v[0], w[1] = v[1], w[2] = v[2];
    } else {
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0));
        w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
    }
}

// The waves' sums of one step, [wave][stream][lane], doubled.
struct Reduce {
    f32x4 v[2][kWaves][2][64];
};

// Steps s0 .. s1 of one entry. w, sc: the two streams' weights and scales at the
// entry's first weight row (stream 1: up, or 16 rows on), `rows` of them, of K
// values; step_rows weight rows from a step to the next; u0, cnt: this
// wave's units of K. b: the rows' values of those units (NB 2: and their
// remainders). done(step, sums of both streams) is called by one wave.
template <int FORM, int NU, int NB, typename Done>
__device__ __forceinline__ void run_steps(const uint8_t* const (&w)[2], const uint8_t* const (&sc)[2], int K, int rows, int step_rows,
                                          int u0, int cnt, int s0, int s1,
                                          const bf16x8 (&b)[NB][NU * Form<FORM>::kLoads * Form<FORM>::kSub], Reduce& red,
                                          int& turn, Done done)
{
    using FM = Form<FORM>;
    constexpr int L = 2 * NU * FM::kLoads, D0 = ring_of(L), U = D0 > L ? D0 / L : 1, D = D0 > L ? U * L : D0;
    static_assert(L % D == 0 || D % L == 0, "ring");
    constexpr bool kScaled = FORM != MOE_W_BF16;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = (uint32_t)FM::bytes(K);
    const uint32_t voff = (uint32_t)r * row_bytes + (uint32_t)u0 * FM::kUnitBytes + 16u * FM::kLoads * g;
    const uint32_t step_bytes = (uint32_t)step_rows * row_bytes, bytes = (uint32_t)rows * row_bytes;
    const uint32_t srow = (uint32_t)(K / 32), svoff = (uint32_t)r * srow + 4u * u0, sstep = (uint32_t)step_rows * srow;
    const uint8_t* const wp[2] = {uni_ptr(w[0]), uni_ptr(w[1])};
    const uint8_t* const sp[2] = {uni_ptr(sc[0]), uni_ptr(sc[1])};

    u32x4 ring[D];
    uint32_t next[U][2][NU];
    // load i of the step `ahead` from s on, into its place in the ring
    auto issue = [&](int place, int s, int ahead, int i) {
        const int u = i / 2 / FM::kLoads, q = i / 2 % FM::kLoads;
        ring[place] = load16(wp[i % 2], s + ahead < s1 && u < cnt ? bytes : 0u, voff,
                             (uint32_t)(s + ahead) * step_bytes + u * FM::kUnitBytes + q * 16);
    };
    auto scales = [&](int place, int s) {
        if constexpr (kScaled)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t records = s < s1 ? (uint32_t)rows * srow : 0u, at = (uint32_t)s * sstep;
                load_words<(NU < 4 ? NU : 4)>(sp[m], records, svoff, at, next[place][m]);
                if constexpr (NU > 4) load_words<NU - 4>(sp[m], records, svoff, at + 16, next[place][m] + 4);
            }
    };
    // (the barriers keep the loads in this order among the products: moved behind
    // them, each wait would be for all of them)
#pragma unroll
    for (int k = 0; k < U; ++k) scales(k, s0 + k);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < D; ++i) {
        issue(i, s0, i / L, i % L);
        __builtin_amdgcn_sched_barrier(0);
    }
    for (int s = s0; s < s1; s += U) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
            uint32_t cur[2][NU];
            if constexpr (kScaled) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < NU; ++i) cur[m][i] = i < cnt ? next[k][m][i] : 0u;  // (past cnt: other rows')
                scales(k, s + k + U);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int m = i % 2, u = i / 2 / FM::kLoads, q = i / 2 % FM::kLoads;
                bf16x8 a[FM::kSub];
                widen<FORM>(ring[(k * L + i) % D], kScaled ? cur[m][u] : 0u, g, a);
#pragma unroll
                for (int j = 0; j < FM::kSub; ++j)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], b[n][(u * FM::kLoads + q) * FM::kSub + j], acc[m], 0, 0, 0);
                issue((k * L + i) % D, s, k + (i + D) / L, (i + D) % L);
                if (m == 1) __builtin_amdgcn_sched_barrier(0);
            }
            if (s + k < s1) {
                red.v[turn][wave][0][lane] = acc[0];
                red.v[turn][wave][1][lane] = acc[1];
                moe::lds::wait_vm_lgkm<63>();  // the sums are in LDS; loads stay in flight
                moe::lds::slot_barrier();
                if (wave == (s + k) % kWaves) {
                    f32x4 a = red.v[turn][0][0][lane], c = red.v[turn][0][1][lane];
#pragma unroll
                    for (int v = 1; v < kWaves; ++v) {
                        a += red.v[turn][v][0][lane];
                        c += red.v[turn][v][1][lane];
                    }
                    done(s + k, a, c);
                }
                turn ^= 1;
            }
        }
    }
}

// Values of an entry's rows as operands: column n = lane % 16 is row n, `row(n)`
// its address, of `width` bf16 values whose units u0 .. u0 + cnt are taken.
template <int FORM, int NU, int N>
__device__ __forceinline__ void load_rows(const uint16_t* row, bool in, int u0, int cnt, bf16x8 (&b)[N])
{
    using FM = Form<FORM>;
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int q = 0; q < FM::kLoads; ++q)
#pragma unroll
            for (int j = 0; j < FM::kSub; ++j) {
                u32x4 v = {0, 0, 0, 0};
                if (in && u < cnt)
                    v = *reinterpret_cast<const u32x4*>(row + (u0 + u) * FM::kUnit + ((g * FM::kLoads + q) * FM::kSub + j) * 8);
                b[(u * FM::kLoads + q) * FM::kSub + j] = __builtin_bit_cast(bf16x8, v);
            }
}

// This workgroup's run of `total` steps.
__device__ __forceinline__ void my_run(int64_t total, int& a, int& z)
{
    a = uni((int)(total * blockIdx.x / gridDim.x));
    z = uni((int)(total * (blockIdx.x + 1) / gridDim.x));
}

// ---------------------------------------------------------------- gate, up --
template <int FORM, int NU>
__global__ __launch_bounds__(kThreads, 2) void few_gateup_kernel(const Few f)
{
    using FM = Form<FORM>;
    __shared__ Tables tab;
    __shared__ Reduce red;
    choose(f, tab, blockIdx.x == 0);
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), n = lane & 15;
    const int per = f.F / kTile, sper = f.SF / kTile, entries = uni(tab.entries), sentries = f.SF ? (f.T + kTile - 1) / kTile : 0;
    const int units = f.H / FM::kUnit, u0 = uni(wave * units / kWaves), cnt = uni((wave + 1) * units / kWaves) - u0;
    int at, end, turn = 0;
    my_run((int64_t)entries * per + (int64_t)sentries * sper, at, end);
    while (at < end) {
        const bool shared = at >= entries * per;
        const int local = shared ? at - entries * per : at, each = shared ? sper : per;
        const int entry = uni(local / each), s0 = local - entry * each, s1 = min(each, s0 + end - at);
        const int e = shared ? 0 : uni((int)tab.entry_e[entry]);
        const int row0 = shared ? entry * kTile : uni((int)tab.entry_row[entry]);
        const int rows = shared ? min(kTile, f.T - row0) : uni((int)tab.entry_n[entry]);
        const size_t first = (size_t)e * f.F;
        const uint8_t* const w[2] = {(shared ? f.sgate : f.gate) + FM::bytes(first * f.H),
                                     (shared ? f.sup : f.up) + FM::bytes(first * f.H)};
        const uint8_t* const sc[2] = {(shared ? f.sgate_s : f.gate_s) + first * (f.H / 32),
                                      (shared ? f.sup_s : f.up_s) + first * (f.H / 32)};
        bf16x8 b[1][NU * FM::kLoads * FM::kSub];
        const int tok = n < rows ? (shared ? row0 + n : (int)tab.tok[row0 + n]) : 0;
        load_rows<FORM, NU>(f.x + (size_t)tok * f.H, n < rows, u0, cnt, b[0]);
        const int width = shared ? f.SF : f.F;
        uint16_t* h = (shared ? f.hs : f.h) + (size_t)(row0 + n) * width + (lane >> 4) * 4;
        run_steps<FORM, NU, 1>(w, sc, f.H, width, kTile, u0, cnt, s0, s1, b, red, turn, [&](int s, const f32x4& g, const f32x4& u) {
            uint32_t hi[2], lo[2];
            float v[4], rest[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = moe::silu(g[i]) * u[i];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                hi[i] = moe::pack_bf16x2(v[2 * i], v[2 * i + 1]);
                rest[2 * i] = v[2 * i] - __uint_as_float(hi[i] << 16);
                rest[2 * i + 1] = v[2 * i + 1] - __uint_as_float(hi[i] & 0xffff0000u);
                lo[i] = moe::pack_bf16x2(rest[2 * i], rest[2 * i + 1]);
            }
            if (n < rows) {
                *reinterpret_cast<uint2*>(h + s * kTile) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(h + f.plane + s * kTile) = make_uint2(lo[0], lo[1]);
            }
        });
        at += s1 - s0;
    }
}

// -------------------------------------------------------------------- down --
template <int FORM, int NU>
__global__ __launch_bounds__(kThreads, 2) void few_down_kernel(const Few f)
{
    using FM = Form<FORM>;
    __shared__ Tables tab;
    __shared__ Reduce red;
    choose(f, tab, false);
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), n = lane & 15;
    const int entries = uni(tab.entries), sentries = f.SF ? (f.T + kTile - 1) / kTile : 0, each = f.H / (2 * kTile);
    int at, end, turn = 0;
    my_run((int64_t)each * (entries * f.parts + sentries * f.sparts), at, end);
    while (at < end) {
        int item = uni(at / each);
        const int s0 = at - item * each, s1 = min(each, s0 + end - at);
        const bool shared = item >= entries * f.parts;
        if (shared) item -= entries * f.parts;
        const int parts = shared ? f.sparts : f.parts, entry = uni(item / parts), part = item - entry * parts;
        const int e = shared ? 0 : uni((int)tab.entry_e[entry]);
        const int row0 = shared ? entry * kTile : uni((int)tab.entry_row[entry]);
        const int rows = shared ? min(kTile, f.T - row0) : uni((int)tab.entry_n[entry]);
        const int K = shared ? f.SF : f.F, units = K / FM::kUnit;
        const int p0 = uni(part * units / parts), pn = uni((part + 1) * units / parts) - p0;
        const int u0 = p0 + uni(wave * pn / kWaves), cnt = p0 + uni((wave + 1) * pn / kWaves) - u0;
        const size_t first = (size_t)e * f.H;
        const uint8_t* base = (shared ? f.sdown : f.down) + FM::bytes(first * K);
        const uint8_t* sbase = (shared ? f.sdown_s : f.down_s) + first * (K / 32);
        const uint8_t* const w[2] = {base, base + FM::bytes((size_t)kTile * K)};
        const uint8_t* const sc[2] = {sbase, sbase + kTile * (K / 32)};
        bf16x8 b[2][NU * FM::kLoads * FM::kSub];
        const uint16_t* h = (shared ? f.hs : f.h) + (size_t)(row0 + (n < rows ? n : 0)) * K;
        load_rows<FORM, NU>(h, n < rows, u0, cnt, b[0]);
        load_rows<FORM, NU>(h + f.plane, n < rows, u0, cnt, b[1]);
        float* y = (shared ? f.ys + (size_t)part * f.T * f.H : f.y + (size_t)part * f.N * f.H) +
                   (size_t)(row0 + n) * f.H + (lane >> 4) * 4;
        run_steps<FORM, NU, 2>(w, sc, K, f.H - kTile, 2 * kTile, u0, cnt, s0, s1, b, red, turn, [&](int s, const f32x4& a, const f32x4& c) {
            if (n < rows) {
                *reinterpret_cast<f32x4*>(y + s * 2 * kTile) = a;
                *reinterpret_cast<f32x4*>(y + s * 2 * kTile + kTile) = c;
            }
        });
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
    const uint16_t *x = static_cast<const uint16_t*>(a.x), *w = static_cast<const uint16_t*>(a.w_router);
    if (s.T <= 1) few_logits_kernel<1><<<s.E, 256, 0, st>>>(s.T, s.H, s.E, x, w, logits);
    else if (s.T <= 2) few_logits_kernel<2><<<s.E, 256, 0, st>>>(s.T, s.H, s.E, x, w, logits);
    else if (s.T <= 4) few_logits_kernel<4><<<s.E, 256, 0, st>>>(s.T, s.H, s.E, x, w, logits);
    else if (s.T <= 8) few_logits_kernel<8><<<s.E, 256, 0, st>>>(s.T, s.H, s.E, x, w, logits);
    else if (s.T <= 16) few_logits_kernel<16><<<s.E, 256, 0, st>>>(s.T, s.H, s.E, x, w, logits);
    else few_logits_kernel<32><<<s.E, 256, 0, st>>>(s.T, s.H, s.E, x, w, logits);
    return hipGetLastError();
}

// Units of K that a wave takes at most, as the kernels' NU.
template <int FORM>
hipError_t launch_form(const Few& f, hipStream_t st)
{
    constexpr int V = FORM == MOE_W_BF16 ? 2 : 1;  // a unit of bf16 is half as long
    const int unit = Form<FORM>::kUnit, grid = cu_count();
    auto waves = [](int units) { return (units + kWaves - 1) / kWaves; };
    const int gu = waves(f.H / unit);
    if (gu <= V) few_gateup_kernel<FORM, V><<<grid, kThreads, 0, st>>>(f);
    else if (gu <= 2 * V) few_gateup_kernel<FORM, 2 * V><<<grid, kThreads, 0, st>>>(f);
    else if (gu <= 4 * V) few_gateup_kernel<FORM, 4 * V><<<grid, kThreads, 0, st>>>(f);
    else if (gu <= 7 * V) few_gateup_kernel<FORM, 7 * V><<<grid, kThreads, 0, st>>>(f);
    else few_gateup_kernel<FORM, 8 * V><<<grid, kThreads, 0, st>>>(f);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    auto part = [&](int K) { return K ? waves((K / unit + moe::few_parts(K) - 1) / moe::few_parts(K)) : 0; };
    const int dn = part(f.F) > part(f.SF) ? part(f.F) : part(f.SF);
    if (dn <= V) few_down_kernel<FORM, V><<<grid, kThreads, 0, st>>>(f);
    else if (dn <= 2 * V) few_down_kernel<FORM, 2 * V><<<grid, kThreads, 0, st>>>(f);
    else few_down_kernel<FORM, 4 * V><<<grid, kThreads, 0, st>>>(f);
    return hipGetLastError();
}

}  // namespace

hipError_t moe_launch_few(const moe_shape_t& s, const MoeFew& a, char* ws, hipStream_t st)
{
    if (s.T == 0) return hipSuccess;
    const moe::FewWsLayout L = moe::few_ws_layout(s, a.shared_F);
    auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
    Few f;
    f.T = s.T, f.H = s.H, f.E = s.E, f.k = s.k, f.F = s.F, f.SF = a.shared_F, f.N = s.T * s.k;
    f.parts = moe::few_parts(s.F), f.sparts = moe::few_parts(a.shared_F);
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
    f.out = static_cast<uint16_t*>(a.out);
    hipError_t e = launch_logits(s, a, logits, st);
    if (e != hipSuccess) return e;
    e = a.form == MOE_W_BF16 ? launch_form<MOE_W_BF16>(f, st)
        : a.form == MOE_W_MX8 ? launch_form<MOE_W_MX8>(f, st) : launch_form<MOE_W_MX4>(f, st);
    if (e != hipSuccess) return e;
    few_combine_kernel<<<dim3((s.H + 1023) / 1024, s.T), 256, 0, st>>>(f);
    return hipGetLastError();
}
