// gemm_mx.hip -- the grouped SwiGLU expert GEMM on 8-bit blocks (serving).
//
//   gate/up: h = blocks(silu(Wg a) * (Wu a)), 32 columns of h to a scale;
//   down:    y = Wd h, rounded to bf16.
//
// Products run on v_mfma_scale_f32_32x32x64_f8f6f4: e4m3 codes with a
// power-of-two scale per 32 values of K, applied inside the instruction, so
// the sums are fp32 sums of the scaled products and no scaling is left for
// the vector unit. Lane l of an operand holds row l % 32; with K cut into
// 16-byte chunks, lanes 0..31 hold chunks 0 and 2 of the 64 and lanes 32..63
// chunks 1 and 3, and the scale of 32-value block b comes from lanes 32 b ..
// 32 b + 31. Weights are the first operand, so a lane's 16 results are one
// token's columns 8 (i / 4) + 4 (l / 32) + i % 4 of a 32-column block.
//
// Expert e's rows are its pieces in rank order (virtual rows), cut into
// tiles; a workgroup of four waves takes one tile of rows and 256 weight rows
// (gate/up: 128 of each), K in stages of 128 bytes through a ring of LDS
// slots that global -> LDS copies fill.
#include "lds_pipe.h"
#include "mx.h"

namespace {

using namespace moe::lds;

constexpr int kThreads = 256;
constexpr int kTN = moe::kMxTileN;
constexpr int kTK = moe::kMxStage;
constexpr int kWBytes = kTN * kTK;       // 32 KB of weights per stage
constexpr int kWCopies = kWBytes / 4096; // 16-byte copies per wave per stage
enum { kGateUp = 0, kDown = 1 };

typedef int i32x8 __attribute__((ext_vector_type(8)));

// schedule (int32): tile_start[E + 1], row_start[E + 1]
__global__ __launch_bounds__(kThreads) void mx_schedule_kernel(int E, int R, int bm, int N,
                                                               const int32_t* __restrict__ plan,
                                                               int32_t* __restrict__ sched,
                                                               int32_t* __restrict__ vrow)
{
    __shared__ int32_t sh[2][kThreads];
    __shared__ int32_t rs[kThreads + 1];
    const moe::PlanLayout L = moe::plan_layout(E, R);
    const int tid = threadIdx.x;
    int c = 0;
    if (tid < E) {
        const int np = plan[L.piece_num + tid];
        for (int p = 0; p < np && p < R; ++p) c += plan[L.piece_cnt + (size_t)tid * R + p];
    }
    sh[0][tid] = (c + bm - 1) / bm;
    sh[1][tid] = c;
    __syncthreads();
    for (int off = 1; off < kThreads; off <<= 1) {
        int a[2];
        for (int q = 0; q < 2; ++q) a[q] = tid >= off ? sh[q][tid - off] : 0;
        __syncthreads();
        for (int q = 0; q < 2; ++q) sh[q][tid] += a[q];
        __syncthreads();
    }
    if (blockIdx.x == 0)
        for (int q = 0; q < 2; ++q) {
            if (tid == 0) sched[q * (E + 1)] = 0;
            if (tid < E) sched[q * (E + 1) + tid + 1] = sh[q][tid];
        }
    if (tid == 0) rs[0] = 0;
    rs[tid + 1] = sh[1][tid];
    __syncthreads();
    const int x = blockIdx.x * kThreads + tid;
    if (x >= N) return;
    int lo = 0, hi = E - 1;  // the expert whose rows hold x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (rs[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    const int v = x - rs[lo];
    const int np = plan[L.piece_num + lo];
    int cum = 0, row = 0;
    for (int p = 0; p < np && p < R; ++p) {
        const int n = plan[L.piece_cnt + (size_t)lo * R + p];
        if (v < cum + n) {
            row = plan[L.piece_row + (size_t)lo * R + p] + (v - cum);
            break;
        }
        cum += n;
    }
    // (rows past the plan's total, or a damaged plan, stay in the buffer)
    vrow[x] = row >= 0 && row < N ? row : 0;
}

__device__ __forceinline__ float fast_silu(float z)
{
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

// Global -> LDS copy of 4 bytes per lane (lane l's land at lds + 4 l) through
// a buffer descriptor, as copy16_or_zero.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy4_or_zero(const void* base, uint32_t voff, uint32_t lds)
{
    const uint64_t b = (uint64_t)(uintptr_t)base;
    i32x4 rsrc;
    rsrc[0] = (int32_t)(uint32_t)b;
    rsrc[1] = (int32_t)(uint32_t)(b >> 32);
    rsrc[2] = (int32_t)kCopyRange;
    rsrc[3] = 0x00020000;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :: "v"(voff), "s"(rsrc), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ i32x8 frag(const char* p0, const char* p1)
{
    const u32x4 a = *reinterpret_cast<const u32x4*>(p0), b = *reinterpret_cast<const u32x4*>(p1);
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// h of one token's 32-column block from the lane's 16 columns (the lane 32
// away holds the other 16): quantised, 16 consecutive codes stored per lane.
__device__ __forceinline__ void store_h(const f32x16& g, const f32x16& u, bool in, uint8_t* dst,
                                        uint8_t* sdst, int half)
{
    float hv[16], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        hv[i] = fast_silu(g[i]) * u[i];
        top = fmaxf(top, moe::mx_abs(hv[i]));
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    const uint32_t byte = moe::mx_scale_byte(top);
    const float inv = moe::mx_inv_scale(byte);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = moe::mx_pack4(hv[4 * i] * inv, hv[4 * i + 1] * inv, hv[4 * i + 2] * inv, hv[4 * i + 3] * inv);
    // w[i] holds columns 8 i + 4 half ..; trade so that half 0 ends up with
    // columns 0..15 and half 1 with 16..31
    const uint32_t give0 = half ? w[0] : w[2], give1 = half ? w[1] : w[3];
    const uint32_t got0 = __shfl_xor(give0, 32), got1 = __shfl_xor(give1, 32);
    const uint4 v = half ? make_uint4(got0, w[2], got1, w[3]) : make_uint4(w[0], got0, w[1], got1);
    if (!in) return;
    *reinterpret_cast<uint4*>(dst + 16 * half) = v;
    if (half == 0) *sdst = (uint8_t)byte;
}

// y of one token's 32-column block: 8 consecutive bf16 columns per store.
__device__ __forceinline__ void store_y(const f32x16& a, bool in, uint16_t* dst, int half, int cols)
{
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = moe::pack_bf16x2(a[2 * i], a[2 * i + 1]);
    // p[2 i], p[2 i + 1]: columns 8 i + 4 half ..; trade quads 2 i and 2 i + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t *e = p + 4 * i, *o = p + 4 * i + 2;  // columns 16 i + ., 16 i + 8 + .
        const uint32_t g0 = half ? e[0] : o[0], g1 = half ? e[1] : o[1];
        const uint32_t r0 = __shfl_xor(g0, 32), r1 = __shfl_xor(g1, 32);
        const uint4 v = half ? make_uint4(r0, r1, o[0], o[1]) : make_uint4(e[0], e[1], r0, r1);
        const int col = 16 * i + 8 * half;
        if (in && col < cols) *reinterpret_cast<uint4*>(dst + col) = v;
    }
}

// One tile: 32 TB rows x 256 weight rows; each wave has all the rows and 64
// of the weight rows (gate/up: 32 gate and the same 32 up).
template <int MODE, int TB>
struct Ring {
    static constexpr int kRows = 32 * TB;
    static constexpr int kA = kRows * kTK;
    static constexpr int kWS = kA + kWBytes;          // weight scales, 4 bytes a row
    static constexpr int kAS = kWS + kTN * 4;         // row scales
    static constexpr int kSlot = (kAS + kRows * 4 + 1023) & ~1023;
    static constexpr int kSlots = 160 * 1024 / kSlot > 4 ? 4 : 160 * 1024 / kSlot;
    static constexpr int kPerStage = kWCopies + TB + 2;  // copies per wave per stage
};

template <int MODE, int TB>
__global__ __launch_bounds__(kThreads, 1) void gemm_mx_kernel(
    int E, int ntiles_n, int H, int F, const uint8_t* __restrict__ a, const uint8_t* __restrict__ as,
    const int32_t* __restrict__ sched, const int32_t* __restrict__ vrow,
    const uint8_t* __restrict__ w0, const uint8_t* __restrict__ s0, const uint8_t* __restrict__ w1,
    const uint8_t* __restrict__ s1, uint8_t* __restrict__ h, uint8_t* __restrict__ hs,
    uint16_t* __restrict__ y)
{
    using RG = Ring<MODE, TB>;
    __shared__ __attribute__((aligned(1024))) char ring[RG::kSlots * RG::kSlot];
    const int tile = blockIdx.x;
    if (tile >= ldc(sched, E) * ntiles_n) return;
    const int tid = threadIdx.x, wave = uni(tid >> 6), lane = tid & 63;
    const int fr = lane & 31, half = lane >> 5;

    // tile -> expert (tile_start), weight tile, rows
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ldc(sched, mid) * ntiles_n <= tile) lo = mid;
        else hi = mid - 1;
    }
    const int e = lo;
    const int mts = ldc(sched, e + 1) - ldc(sched, e);
    const int local = tile - ldc(sched, e) * ntiles_n;
    const int nt = local / mts, v0 = local % mts * RG::kRows;
    const int x0 = ldc(sched, E + 1 + e) + v0;
    const int rows = min(RG::kRows, ldc(sched, E + 1 + e + 1) - x0);
    const int n0 = nt * (MODE == kGateUp ? kTN / 2 : kTN);
    const int K = MODE == kGateUp ? H : F, KT = K / kTK, KS = K / moe::kMxBlock;
    const int wrows = MODE == kGateUp ? F : H;

    // copy sources (see lds_pipe.h): instruction q = wave + 4 i fills rows
    // 8 q .. 8 q + 7 of an operand, lane l row 8 q + l / 8, chunk l % 8
    const char* abase = MODE == kGateUp ? (const char*)a : (const char*)a + (size_t)x0 * K;
    const char* asbase = MODE == kGateUp ? (const char*)as : (const char*)as + (size_t)x0 * KS;
    const char* wb0 = (const char*)w0 + (size_t)e * F * H;
    const char* wb1 = MODE == kGateUp ? (const char*)w1 + (size_t)e * F * H : wb0;
    const char* sb0 = (const char*)s0 + (size_t)e * F * (H / moe::kMxBlock);
    const char* sb1 = MODE == kGateUp ? (const char*)s1 + (size_t)e * F * (H / moe::kMxBlock) : sb0;
    if (MODE == kDown) sb0 = sb1 = (const char*)s0 + (size_t)e * H * (F / moe::kMxBlock);
    auto source_row = [&](int r) { return MODE == kGateUp ? (uint32_t)vrow[x0 + r] : (uint32_t)r; };
    uint32_t aoff[TB], woff[kWCopies];
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        const int r = 8 * (wave + 4 * i) + (lane >> 3);
        aoff[i] = r < rows ? source_row(r) * (uint32_t)K + (uint32_t)(((lane & 7) ^ swz(r)) * 16) : kZeroRow;
    }
    auto weight_row = [&](int r) {
        return (uint32_t)(MODE == kGateUp ? n0 + (r & 127) : min(n0 + r, wrows - 1));
    };
#pragma unroll
    for (int i = 0; i < kWCopies; ++i) {
        const int r = 8 * (wave + 4 * i) + (lane >> 3);
        woff[i] = weight_row(r) * (uint32_t)K + (uint32_t)(((lane & 7) ^ swz(r)) * 16);
    }
    // scales: wave w copies 4 bytes of weight rows 64 w + lane and of tile
    // rows 8 TB w + lane (lanes below 8 TB)
    const int ar = 8 * TB * wave + lane;
    const uint32_t asoff = lane < 8 * TB && ar < rows ? source_row(ar) * (uint32_t)KS : kZeroRow;
    const uint32_t wsoff = weight_row(64 * wave + lane) * (uint32_t)KS;
    const uint32_t ring_u = (uint32_t)(uintptr_t)ring;
    auto copy_stage = [&](int st) {
        const uint32_t slot = ring_u + (uint32_t)(st % RG::kSlots) * RG::kSlot;
        const int kb = st * kTK;
#pragma unroll
        for (int i = 0; i < TB; ++i) copy16_or_zero(abase + kb, aoff[i], slot + wave * 1024 + i * 4096);
#pragma unroll
        for (int i = 0; i < kWCopies; ++i)
            copy16((i < 4 ? wb0 : wb1) + kb, woff[i], slot + RG::kA + wave * 1024 + i * 4096);
        copy4_or_zero((wave < 2 ? sb0 : sb1) + st * 4, wsoff, slot + RG::kWS + wave * 256);
        if (lane < 8 * TB) copy4_or_zero(asbase + st * 4, asoff, slot + RG::kAS + wave * 32 * TB);
    };

    f32x16 acc[TB][2];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[b][j][q] = 0.0f;
    // weight row of this wave's block j
    auto wrow = [&](int j) { return MODE == kGateUp ? 32 * wave + 128 * j + fr : 64 * wave + 32 * j + fr; };

    constexpr int kAhead = RG::kSlots - 1;
    for (int st = 0; st < kAhead && st < KT; ++st) copy_stage(st);
    for (int s = 0; s < KT; ++s) {
        // stage s landed in this wave: only copies of later stages are out
        const int after = min(KT - 1, s + kAhead - 1) - s;
        if (after >= 2) wait_vm_lgkm<2 * RG::kPerStage>();
        else if (after == 1) wait_vm_lgkm<RG::kPerStage>();
        else wait_vm_lgkm<0>();
        slot_barrier();  // ... in every wave; and stage s - 1's slot is free
        if (s + kAhead < KT) copy_stage(s + kAhead);
        const char* slot = ring + (s % RG::kSlots) * RG::kSlot;
        int ws[2], ts[TB];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            ws[j] = (int)(*reinterpret_cast<const uint32_t*>(slot + RG::kWS + wrow(j) * 4) >> (8 * half));
#pragma unroll
        for (int b = 0; b < TB; ++b)
            ts[b] = (int)(*reinterpret_cast<const uint32_t*>(slot + RG::kAS + (32 * b + fr) * 4) >> (8 * half));
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int c0 = ((4 * kk + half) ^ swz(fr)) * 16, c1 = ((4 * kk + 2 + half) ^ swz(fr)) * 16;
            i32x8 wf[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const char* p = slot + RG::kA + wrow(j) * 128;
                wf[j] = frag(p + c0, p + c1);
            }
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const char* p = slot + (32 * b + fr) * 128;
                const i32x8 tf = frag(p + c0, p + c1);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[b][j] = kk == 0
                        ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[j], tf, acc[b][j], 0, 0, 0, ws[j], 0, ts[b])
                        : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[j], tf, acc[b][j], 0, 0, 2, ws[j], 2, ts[b]);
            }
        }
    }

#pragma unroll
    for (int b = 0; b < TB; ++b) {
        const int row = 32 * b + fr;
        const bool in = row < rows;
        if (MODE == kGateUp) {
            const int col = n0 + 32 * wave;
            const size_t x = (size_t)x0 + (in ? row : 0);
            store_h(acc[b][0], acc[b][1], in, h + x * F + col, hs + x * (F / moe::kMxBlock) + col / moe::kMxBlock, half);
        } else {
            uint16_t* dst = y + (size_t)vrow[x0 + (in ? row : 0)] * H;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = n0 + 64 * wave + 32 * j;
                store_y(acc[b][j], in, dst + col, half, H - col);
            }
        }
    }
}

constexpr int kTB = 2;

}  // namespace

hipError_t moe_launch_grouped_gemm_mx(const moe_shape_t& s, const void* a, const void* a_s,
                                      const int32_t* plan, const MoeMxWeights& w, void* y,
                                      char* ws, hipStream_t st)
{
    const int N = s.T * s.k;
    if (N == 0) return hipSuccess;
    const moe::MxWsLayout W = moe::mx_ws_layout(s);
    int32_t* sched = reinterpret_cast<int32_t*>(ws + W.sched);
    int32_t* vrow = reinterpret_cast<int32_t*>(ws + W.vrow);
    uint8_t *h = reinterpret_cast<uint8_t*>(ws + W.h), *hs = reinterpret_cast<uint8_t*>(ws + W.hs);
    const uint8_t *av = static_cast<const uint8_t*>(a), *asv = static_cast<const uint8_t*>(a_s);
    const int bm = 32 * kTB;
    mx_schedule_kernel<<<(N + kThreads - 1) / kThreads, kThreads, 0, st>>>(s.E, s.R, bm, N, plan, sched, vrow);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t mt = N / bm + (s.E < N ? s.E : N);
    int nt = s.F / (kTN / 2);
    gemm_mx_kernel<kGateUp, kTB><<<(int)(mt * nt), kThreads, 0, st>>>(
        s.E, nt, s.H, s.F, av, asv, sched, vrow, w.gate, w.gate_s, w.up, w.up_s, h, hs, nullptr);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    nt = (s.H + kTN - 1) / kTN;
    gemm_mx_kernel<kDown, kTB><<<(int)(mt * nt), kThreads, 0, st>>>(
        s.E, nt, s.H, s.F, h, hs, sched, vrow, w.down, w.down_s, nullptr, nullptr, nullptr, nullptr,
        static_cast<uint16_t*>(y));
    return hipGetLastError();
}
