// Decode over the 8-bit key/value cache: n new query tokens per sequence (one, or a
// few drafted ones to verify), windowed attention for each and whole-prefix attention
// for sequences with a token whose gate passes the threshold.
//
// Sources: "Learning When to Attend", "Empirical Validation and System Optimization"
// (the savings carry over to time-to-first-token and token generation, the skipped
// work being memory-bound global reads); "LoGo: Token-Level Dynamic Local-Global
// Attention", Abstract (a gate decides per token, a threshold controller keeps the
// share).
//
// Bound by HBM: one byte per element of the cache read, about 2 R FLOP per byte for
// the R = (Hq / Hkv) n query rows that share a key/value head.
//   decode8_partial_kernel  one wave of persistent warps.  The work is a list of
//     units: for every (sequence, key/value head) the 64-position stages before the
//     window (only where a token is global), then the stages that reach into it.
//     The list is cut into equal shares, one per warp, so every warp reads the same
//     number of bytes whatever the lengths and gates are; the lengths are read on the
//     device.  A warp streams its stages through a private ring in shared memory,
//     filled by TMA (rows swizzled), tracked by one mbarrier per stage and kept full
//     from one sequence to the next.  Per stage:
//       S^T = K q^T   mma.sync m16n8k16, fp16 in, fp32 out: positions are the rows,
//                     the query rows the columns.  Codes become fp16 exactly.  The
//                     order of the head dimension inside a product is free, so a lane
//                     uses the four consecutive codes that ldmatrix gives it as they
//                     are, and q is stored in that order.
//       softmax       online, fp32, one maximum per stage and query row;
//       O^T += V^T P^T  V^T by ldmatrix.trans on pairs of codes: a word holds two
//                     head-dimension columns at two positions, and one byte permute
//                     sorts it into the fp16 pairs of two rows of V^T.  Each stage's
//                     product starts from zero and joins O with the stage's V scale in
//                     fp32, so scales of any ratio meet only in 32 bits.
//     Positions outside the window and inside it go to separate partial states
//     (m, l, o): a position is read once, local attention is the inside state, global
//     attention both.
//   decode8_combine_kernel  one CTA per query row: joins the states of the warps that
//     held a share of the row's stages; o = local + sigmoid(g) * global, one rounding.
//
// mma.sync and not tcgen05: a stage of 16 KB takes an SM about 700 cycles to fetch and
// its 64 products a fraction of that, and codes need a conversion in registers, which
// an operand read from shared memory by tcgen05 would not see.
//
// Roundings: q is scaled by a power of two per row, so that its largest element lies
// in [2^14, 2^15), and rounded to fp16 (exact for elements down to 2^-28 of the
// largest).  P is 2^15 exp2(s - m) in fp16: 11 bits, 3 more than bf16, with values
// down to 2^-39 of the largest kept.  The sum l uses the unrounded P.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cache8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace logo {

namespace {

#ifndef LOGO_DEC8_WARPS
#define LOGO_DEC8_WARPS 6
#endif
#ifndef LOGO_DEC8_STAGES
#define LOGO_DEC8_STAGES 2
#endif
#ifndef LOGO_DEC8_KUNROLL
#define LOGO_DEC8_KUNROLL 2
#endif
#ifndef LOGO_DEC8_KUNROLL
#define LOGO_DEC8_KUNROLL 2
#endif
constexpr int kKUnroll = LOGO_DEC8_KUNROLL;  // of the loop over head-dimension pairs of the scores
constexpr float kPBias = 15.f;  // P is held times 2^15: the state's m is the maximum less 15

template <int D, int NT>
struct D8 {
    static constexpr int kTile = kDec8Stage * D;                  // codes of K (or V) of one stage, bytes
    static constexpr int kStageBytes = 2 * kTile;                 // K then V
    static constexpr int kStages = LOGO_DEC8_STAGES * 128 / D;    // ring depth: the same bytes for both D
    static constexpr int kRingBytes = kStages * kStageBytes;
    static constexpr int kQBytes = (D / 16) * NT * 32 * 8;        // q fragments of one warp
    static constexpr int kWarpBytes = kRingBytes + (kQBytes + 1023) / 1024 * 1024;
    static constexpr int kWarps = NT == 4 ? LOGO_DEC8_WARPS - 1 : LOGO_DEC8_WARPS;  // independent warps per CTA
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kSmem = kWarps * kWarpBytes + 1024;      // + alignment slack
    static constexpr int MT = NT == 4 ? 2 : 4;                    // 16-position tiles per softmax step
};

// ---------------------------------------------------------------- the list of units

// Units of one sequence: `out` stages before the window ([0, out), sequences with a
// global token only), then stages [in0, in1).  They overlap in the stages that the
// first window edges of the n tokens cross.
struct Plan {
    int len;   // 0 also for an invalid length
    int out, in0, in1;
    __device__ int units() const { return out + in1 - in0; }
};

__device__ __forceinline__ bool takes_global(float g, float tau) { return g > tau; }  // false for NaN

// Every load is issued before the first is used: they do not depend on one another.
__device__ __forceinline__ Plan plan_of(const Decode8Params& p, int b)
{
    Plan pl{0, 0, 0, 0};
    const int len = p.cache_len[b];
    const float tau = *p.tau;
    bool any = false;
    for (int i = 0; i < p.n; ++i) any |= takes_global(p.gate[(long long)b * p.n + i], tau) && i >= p.n - len;
    if (len <= 0 || len > p.Lmax) return pl;
    // window edges of the first and last token
    const int e0 = len - p.n - p.W + 1, e1 = len - p.W;
    pl.len = len;
    pl.in0 = e0 > 0 ? e0 / kDec8Stage : 0;
    pl.in1 = (len + kDec8Stage - 1) / kDec8Stage;
    pl.out = any && e1 > 0 ? (e1 + kDec8Stage - 1) / kDec8Stage : 0;
    return pl;
}

__device__ __forceinline__ int warp_scan(int x)  // inclusive
{
    const int lane = threadIdx.x & 31;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// T units cut into N shares: the first `rest` warps take one unit more than the others.
// T fits 32 bits: a unit is at least 8 KB of cache, read at most twice.
struct Shares {
    int N, each, rest;
    __device__ __forceinline__ Shares(int T, int most, int least)
    {
        const int w = (T + least - 1) / least;  // a share is worth its partial state
        N = w < most ? w : most;
        each = N ? T / N : 0;
        rest = N ? T % N : 0;
    }
    __device__ __forceinline__ int first(int w) const { return w * each + (w < rest ? w : rest); }
    __device__ __forceinline__ int warp_of(int u) const
    {
        const int big = rest * (each + 1);
        return u < big ? u / (each + 1) : rest + (u - big) / each;
    }
};

// Fewest units of a share, by the column tiles that a partial state spans.
__host__ __device__ constexpr int least_units(int nt) { return nt; }

// Partial states: slot (warp + pair) is unique, since along the list either the warp
// or the pair (sequence, key/value head) moves on from one share to the next.  A slot
// holds R rows for each kind (0: inside the window, 1: before it): (m, l) and o apart.
__host__ __device__ inline long long slots8(long long pairs) { return kDec8MaxWarps + pairs; }
__device__ __forceinline__ long long row_at(const Decode8Params& p, int warp, int pair, int kind)
{
    return (((long long)warp + pair) * 2 + kind) * p.R;
}
__device__ __forceinline__ float2* part_ml(const Decode8Params& p) { return reinterpret_cast<float2*>(p.part); }
__device__ __forceinline__ float* part_o(const Decode8Params& p)
{
    return p.part + slots8((long long)p.B * p.Hkv) * 2 * p.R * 2;
}

// ---------------------------------------------------------------- fragments

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ uint32_t movm(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// D(16x8, fp32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The codes in bytes 0, 1 (-> lo) and 2, 3 (-> hi) of a word as fp16 pairs, exact.
template <int TYPE>
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    if (TYPE == kCacheE4M3) {
        asm("{\n\t.reg .b16 x, y;\n\t"
            "mov.b32 {x, y}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, x;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // 0x6400 | u is 1024 + u in fp16 for u in [0, 255]; u = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));  // 1152
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
    }
}

// A word of ldmatrix.trans holds two positions' codes of columns 2g and 2g + 1: bytes
// (pos 0: 2g, 2g + 1; pos 1: 2g, 2g + 1).  As fp16 pairs over the positions: column 2g, column 2g + 1.
template <int TYPE>
__device__ __forceinline__ void to_f16_pairs(uint32_t w, uint32_t& even, uint32_t& odd)
{
    if (TYPE == kCacheE4M3) {
        to_f16<TYPE>(__byte_perm(w, 0u, 0x3120), even, odd);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4240), b = __byte_perm(u, 0x64646464u, 0x4341);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"(a), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(b), "r"(0x64806480u));
    }
}

// Address of the 16-byte unit u of row r in a tile of D-byte rows that TMA wrote with
// the swizzle of that row length (128B: unit ^ row mod 8; 64B: unit ^ (row / 2) mod 4).
template <int D>
__device__ __forceinline__ uint32_t swz(uint32_t tile, int r, int u)
{
    return D == 128 ? tile + r * 128 + (((u ^ r) & 7) << 4) : tile + r * 64 + (((u ^ (r >> 1)) & 3) << 4);
}

// ---------------------------------------------------------------- one warp's work

struct Ring8 {
    uint32_t base;   // shared address of stage 0
    uint64_t* full;  // one barrier per stage
    uint32_t issued, used;
};

// Softmax state of the warp's query rows.  Lane (g, t) = (lane / 4, lane % 4) has
// columns 8 nt + 2t + c (c = 0, 1): their maxima (shared by the 8 lanes of the same
// t), a share of their sums, and of O^T the rows 16 u + 2g + h at o[u][nt][2h + c].
template <int D, int NT>
struct State8 {
    float m[NT][2], l[NT][2];
    float o[D / 16][NT][4];
    __device__ __forceinline__ void init()
    {
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
        #pragma unroll
        for (int u = 0; u < D / 16; ++u)
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                #pragma unroll
                for (int e = 0; e < 4; ++e) o[u][nt][e] = 0.f;
    }
};

template <int D, int NT>
__device__ __forceinline__ void store_state8(const Decode8Params& p, const State8<D, NT>& st, long long row)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        #pragma unroll
        for (int c = 0; c < 2; ++c) {
            float l = st.l[nt][c];
            #pragma unroll
            for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
            const int r = 8 * nt + 2 * t + c;
            if (r >= p.R) continue;
            if (g == 0) part_ml(p)[row + r] = make_float2(st.m[nt][c], l);
            float* o = part_o(p) + (row + r) * D + 2 * g;
            #pragma unroll
            for (int u = 0; u < D / 16; ++u)
                *reinterpret_cast<float2*>(o + 16 * u) = make_float2(st.o[u][nt][c], st.o[u][nt][2 + c]);
        }
    }
}

// Where in the list a warp is: unit `off` of key/value head hk of sequence b.
struct Cursor {
    int b, hk, off, units;
    Plan pl;
    __device__ __forceinline__ int pair(int Hkv) const { return b * Hkv + hk; }
    __device__ __forceinline__ int stage() const { return off < pl.out ? off : off - pl.out + pl.in0; }
    __device__ __forceinline__ void next_pair(const Decode8Params& p)
    {
        off = 0;
        if (++hk < p.Hkv) return;
        hk = 0;
        do {
            if (++b >= p.B) return;
            pl = plan_of(p, b);
        } while (pl.units() == 0);
        units = pl.units();
    }
    __device__ __forceinline__ void next(const Decode8Params& p)
    {
        if (++off == units) next_pair(p);
    }
};

// The next unit's keys and values into the ring (all lanes keep count, lane 0 copies).
template <int D, int NT>
__device__ __forceinline__ void issue_unit(const Decode8Params& p, Ring8& ring, Cursor& at)
{
    using G = D8<D, NT>;
    if ((threadIdx.x & 31) == 0) {
        const uint32_t s = ring.issued % G::kStages;
        uint8_t* dst = reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(ring.base + s * G::kStageBytes));
        const int row = at.stage() * kDec8Stage, slab = at.pair(p.Hkv);
        fence_proxy_async_smem();  // the warp's reads of this stage come before the copy engine's writes
        mbar_arrive_expect_tx(&ring.full[s], G::kStageBytes);
        tma_load_3d(dst, &p.tm_k, &ring.full[s], 0, row, slab, policy_evict_first());
        tma_load_3d(dst + G::kTile, &p.tm_v, &ring.full[s], 0, row, slab, policy_evict_first());
    }
    ++ring.issued;
    at.next(p);
}

// Per-lane constants of the (sequence, key/value head) at hand.
template <int NT>
struct Rows8 {
    float qf[NT][2];  // scale * log2(e) / (the power of two in the row's fp16 q)
    int tok[NT][2];   // the column's token
};

// q of one (sequence, key/value head) to fp16 in shared memory, in fragment order: lane
// (g, t) of unit kk, tile nt holds row 8 nt + g, elements 16 kk + 4t .. + 3.
template <int D, int NT>
__device__ __forceinline__ void stage_q(const Decode8Params& p, long long pair, uint2* qs, Rows8<NT>& rw)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint16_t* q = p.q + pair * p.R * D + 4 * t;
    __syncwarp();
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + g;
        uint2 w[D / 16];
        uint32_t big = 0;
        #pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            w[kk] = r < p.R ? *reinterpret_cast<const uint2*>(q + (long long)r * D + 16 * kk) : make_uint2(0u, 0u);
        #pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            big = __vmaxu2(big, __vmaxu2(w[kk].x & 0x7fff7fffu, w[kk].y & 0x7fff7fffu));
        big = max(big & 0xffffu, big >> 16);
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        int ex = 141 - (int)(big >> 7);  // largest element into [2^14, 2^15)
        ex = ex > 127 ? 127 : ex;
        const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
        #pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint2 f;
            f.x = pack_f16x2(__uint_as_float(w[kk].x << 16) * up, __uint_as_float(w[kk].x & 0xffff0000u) * up);
            f.y = pack_f16x2(__uint_as_float(w[kk].y << 16) * up, __uint_as_float(w[kk].y & 0xffff0000u) * up);
            qs[(kk * NT + nt) * 32 + lane] = f;
        }
        #pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int e2 = __shfl_sync(0xffffffffu, ex, 4 * (2 * t + c));
            rw.qf[nt][c] = ldexpf(p.scale_log2, -e2);
            rw.tok[nt][c] = (8 * nt + 2 * t + c) % p.n;
        }
    }
    __syncwarp();
}

// A stage that some column sees in part (positions pos0 .., token i sees [lo0 + i, hi0 + i],
// from 0 on where that is negative): values at positions that no column sees are made
// zero in shared memory, whatever the cache holds there (their P is zero, but zero times
// NaN is not).  Says whether an e4m3 NaN is left at a position that only some tokens see.
template <int TYPE, int D>
__device__ __noinline__ bool mask_values(uint32_t tileV, int pos0, int lo0, int hi0, int n)
{
    const int lane = threadIdx.x & 31;
    uint8_t* v = reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(tileV));
    const int last = hi0 + n - 1;
    bool nan = false;
    #pragma unroll 1
    for (int k = lane; k < kDec8Stage * D / 16; k += 32) {
        const int pos = pos0 + k / (D / 16);
        uint4* at = reinterpret_cast<uint4*>(v + 16 * k);
        if (pos < lo0 || pos > last) {
            *at = make_uint4(0u, 0u, 0u, 0u);
        } else if (TYPE == kCacheE4M3 && (pos < lo0 + n - 1 || pos > hi0)) {
            const uint4 w = *at;
            auto has = [](uint32_t x) { return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u; };
            nan |= has(w.x) || has(w.y) || has(w.z) || has(w.w);
        }
    }
    __syncwarp();
    return __any_sync(0xffffffffu, nan);
}

// Such NaN codes go straight into the output of the tokens that see them, and are made zero.
template <int D, int NT>
__device__ __forceinline__ void place_nan(uint32_t tileV, int pos0, int lo0, int hi0, int n, const Rows8<NT>& rw,
                                          State8<D, NT>& st)
{
    const int lane = threadIdx.x & 31, g = lane >> 2;
    uint8_t* v = reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(tileV));
    #pragma unroll 1
    for (int r = 0; r < kDec8Stage; ++r) {
        const int pos = pos0 + r;
        if (pos < lo0 || pos > hi0 + n - 1 || (pos >= lo0 + n - 1 && pos <= hi0)) continue;  // seen by none or by all
        #pragma unroll
        for (int u = 0; u < D / 16; ++u) {
            uint16_t* at = reinterpret_cast<uint16_t*>(v + (swz<D>(tileV, r, u) - tileV) + 2 * g);
            const uint32_t w = *at;
            const bool nan0 = (w & 0x7fu) == 0x7fu, nan1 = (w & 0x7f00u) == 0x7f00u;
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                #pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const bool sees = pos >= lo0 + rw.tok[nt][c] && pos <= hi0 + rw.tok[nt][c];
                    if (sees && nan0) st.o[u][nt][c] = __int_as_float(0x7fffffff);
                    if (sees && nan1) st.o[u][nt][2 + c] = __int_as_float(0x7fffffff);
                }
            __syncwarp();  // four lanes share a word
            *at = (uint16_t)((nan0 ? 0u : w & 0xffu) | (nan1 ? 0u : w & 0xff00u));
        }
    }
    __syncwarp();
}

// One stage: scores, softmax step, products.  `masked`: some column sees it in part.
template <int TYPE, int D, int NT>
__device__ __forceinline__ void do_stage(State8<D, NT>& st, const Rows8<NT>& rw, const uint2* qs, uint32_t tileK,
                                         float ks, float vs, bool masked, int pos0, int lo0, int hi0, int n)
{
    using G = D8<D, NT>;
    constexpr int MT = G::MT, kSteps = 4 / MT;
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int kr = (lane & 7) + 8 * ((lane >> 3) & 1), ku = lane >> 4;  // ldmatrix roles: row, 16-byte unit
    const uint32_t tileV = tileK + G::kTile;
    if (masked && mask_values<TYPE, D>(tileV, pos0, lo0, hi0, n) && TYPE == kCacheE4M3)
        place_nan<D, NT>(tileV, pos0, lo0, hi0, n, rw, st);
    #pragma unroll 1
    for (int step = 0; step < kSteps; ++step) {
        const int row0 = step * 16 * MT;
        // S^T = K q^T: rows = positions 16 mt + g (+ 8), columns = query rows
        float sc[MT][NT][4];
        #pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                #pragma unroll
                for (int x = 0; x < 4; ++x) sc[mt][nt][x] = 0.f;
        #pragma unroll kKUnroll
        for (int kk = 0; kk < D / 32; ++kk) {
            uint2 b0[NT], b1[NT];
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                b0[nt] = qs[((2 * kk) * NT + nt) * 32 + lane];
                b1[nt] = qs[((2 * kk + 1) * NT + nt) * 32 + lane];
            }
            #pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t w[4], x[4], y[4];
                ldsm4(swz<D>(tileK, row0 + 16 * mt + kr, 2 * kk + ku), w);
                #pragma unroll
                for (int q = 0; q < 4; ++q) to_f16<TYPE>(w[q], x[q], y[q]);
                #pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(sc[mt][nt], x[0], x[1], y[0], y[1], b0[nt].x, b0[nt].y);
                    mma_f16(sc[mt][nt], x[2], x[3], y[2], y[3], b1[nt].x, b1[nt].y);
                }
            }
        }
        // online softmax
        uint32_t pb[MT][NT][2];
        float al[NT][2];
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            #pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float f = ks * rw.qf[nt][c];
                #pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) sc[mt][nt][2 * h + c] *= f;
                if (masked) {
                    const int lo = lo0 + rw.tok[nt][c] - pos0 - row0 - g, hi = hi0 + rw.tok[nt][c] - pos0 - row0 - g;
                    #pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        #pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (16 * mt + 8 * h < lo || 16 * mt + 8 * h > hi) sc[mt][nt][2 * h + c] = -INFINITY;
                }
                float mx = -INFINITY;
                #pragma unroll
                for (int mt = 0; mt < MT; ++mt) mx = fmax3(mx, sc[mt][nt][c], sc[mt][nt][2 + c]);
                #pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float mn = fmaxf(st.m[nt][c], mx - kPBias);
                const float r = mn == -INFINITY ? 0.f : mn;
                al[nt][c] = fast_exp2(st.m[nt][c] - r);  // 0 while nothing was seen
                st.m[nt][c] = mn;
                float sum = 0.f;
                #pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x = fast_exp2(sc[mt][nt][2 * h + c] - r);
                        sc[mt][nt][2 * h + c] = x;
                        sum += x;
                    }
                st.l[nt][c] = fmaf(st.l[nt][c], al[nt][c], sum);
            }
            // P^T fragments: the score fragment's 8x8 quarters transposed in registers
            #pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                #pragma unroll
                for (int h = 0; h < 2; ++h)
                    pb[mt][nt][h] = movm(pack_f16x2(sc[mt][nt][2 * h], sc[mt][nt][2 * h + 1]));
        }
        // O^T = O^T alpha + (V^T P^T) vs
        #pragma unroll
        for (int u = 0; u < D / 16; ++u) {
            float acc[NT][4];
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                #pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
            #pragma unroll
            for (int h = 0; h < MT / 2; ++h) {
                uint32_t w[4], ev[4], od[4];
                ldsm4t(swz<D>(tileV, row0 + 32 * h + lane, u), w);
                #pragma unroll
                for (int i = 0; i < 4; ++i) to_f16_pairs<TYPE>(w[i], ev[i], od[i]);
                #pragma unroll
                for (int k = 0; k < 2; ++k)
                    #pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(acc[nt], ev[2 * k], od[2 * k], ev[2 * k + 1], od[2 * k + 1], pb[2 * h + k][nt][0],
                                pb[2 * h + k][nt][1]);
            }
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                #pragma unroll
                for (int e = 0; e < 4; ++e)
                    st.o[u][nt][e] = fmaf(acc[nt][e], vs, st.o[u][nt][e] * al[nt][e & 1]);
        }
    }
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(D8<D, NT>::kThreads, 1) decode8_partial_kernel(const __grid_constant__ Decode8Params p)
{
    using G = D8<D, NT>;
    extern __shared__ uint8_t dsmem8[];
    __shared__ uint64_t full_bars[G::kWarps][G::kStages];
    __shared__ int abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Let the combine kernel's CTAs be placed; they wait for this grid's end before they read.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t was = *reinterpret_cast<volatile uint32_t*>(p.status);
    if (lane == 0) {
        for (int s = 0; s < G::kStages; ++s) mbar_init(&full_bars[warp][s], 1);
        fence_barrier_init();
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    // The whole list's length (every warp for itself).
    int T = 0;
    bool bad = false;
    for (int b = lane; b - lane < p.B; b += 32) {
        Plan pl{0, 0, 0, 0};
        if (b < p.B) {
            pl = plan_of(p, b);
            bad |= pl.len == 0 && p.cache_len[b] != 0;
        }
        T += (int)__reduce_add_sync(0xffffffffu, pl.units()) * p.Hkv;
    }
    if (bad && blockIdx.x == 0 && warp == 0) atomicOr(p.status, kStatusBadArgument);
    if (threadIdx.x == 0) abort_word = (was & kStatusTimeout) ? 1 : 0;
    __syncthreads();
    volatile int* abort_flag = &abort_word;
    if (*abort_flag) return;
    const Shares sh(T, (int)gridDim.x * G::kWarps, least_units(NT));
    const int gw = warp * (int)gridDim.x + (int)blockIdx.x;  // few shares: one per SM first
    if (gw >= sh.N) return;
    int left = sh.first(gw + 1) - sh.first(gw);
    Cursor at{};
    {
        int before = sh.first(gw);  // units ahead of the share, less those of the sequences passed
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const Plan mine = b0 + lane < p.B ? plan_of(p, b0 + lane) : Plan{0, 0, 0, 0};
            const int incl = warp_scan(mine.units()) * p.Hkv;
            const unsigned past = __ballot_sync(0xffffffffu, incl > before);
            if (past == 0) {
                before -= __shfl_sync(0xffffffffu, incl, 31);
                continue;
            }
            const int src = __ffs(past) - 1;
            at.b = b0 + src;
            at.pl.len = __shfl_sync(0xffffffffu, mine.len, src);
            at.pl.out = __shfl_sync(0xffffffffu, mine.out, src);
            at.pl.in0 = __shfl_sync(0xffffffffu, mine.in0, src);
            at.pl.in1 = __shfl_sync(0xffffffffu, mine.in1, src);
            at.units = at.pl.units();
            before -= __shfl_sync(0xffffffffu, incl, src) - at.units * p.Hkv;
            at.hk = before / at.units;
            at.off = before % at.units;
            break;
        }
    }
    const uint32_t base = ((smem_u32(dsmem8) + 1023u) & ~1023u) + warp * G::kWarpBytes;
    uint2* qs = reinterpret_cast<uint2*>(__cvta_shared_to_generic(base + G::kRingBytes));
    Ring8 ring{base, full_bars[warp], 0, 0};
    Cursor ahead = at;
    int to_issue = left;
    for (int i = 0; i < G::kStages && to_issue > 0; ++i, --to_issue) issue_unit<D, NT>(p, ring, ahead);
    Rows8<NT> rw;
    State8<D, NT> st;
    int staged = -1;
    bool ok = true;
    while (left > 0 && ok) {
        // A run: stages of one pair and one kind, ended by the kind's last stage or the share's.
        const int pair = at.pair(p.Hkv);
        const bool inside = at.off >= at.pl.out;
        const int stage0 = at.stage(), most = (inside ? at.units : at.pl.out) - at.off, cnt = left < most ? left : most;
        // token i sees [lo0 + i, hi0 + i]: its window, or what lies before it
        const int lo0 = inside ? at.pl.len - p.n - p.W + 1 : -kDec8MaxRows;  // at most 0 for every token
        const int hi0 = at.pl.len - p.n - (inside ? 0 : p.W);
        const float* ksp = p.k_scale + (long long)pair * p.nblk;
        const float* vsp = p.v_scale + (long long)pair * p.nblk;
        float ks32 = 0.f, vs32 = 0.f;  // scales of 32 stages, one per lane
        if (lane < cnt) {
            ks32 = ksp[(stage0 + lane) / p.block_units];
            vs32 = vsp[(stage0 + lane) / p.block_units];
        }
        if (pair != staged) stage_q<D, NT>(p, pair, qs, rw);
        staged = pair;
        st.init();
        for (int i = 0; i < cnt; ++i) {
            if ((i & 31) == 0 && i > 0) {
                const int blk = (stage0 + i + lane) / p.block_units;
                ks32 = i + lane < cnt ? ksp[blk] : 0.f;
                vs32 = i + lane < cnt ? vsp[blk] : 0.f;
            }
            const float ks = __shfl_sync(0xffffffffu, ks32, i & 31), vs = __shfl_sync(0xffffffffu, vs32, i & 31);
            const uint32_t s = ring.used % G::kStages;
            ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[s], (ring.used / G::kStages) & 1, abort_flag, p.status,
                                                   p.timeout_ns));
            if (!ok) break;
            const int pos0 = (stage0 + i) * kDec8Stage;
            const bool masked = pos0 < lo0 + p.n - 1 || pos0 + kDec8Stage - 1 > hi0;
            do_stage<TYPE, D, NT>(st, rw, qs, ring.base + s * G::kStageBytes, ks, vs, masked, pos0, lo0, hi0, p.n);
            ++ring.used;
            __syncwarp();
            if (to_issue > 0) {
                issue_unit<D, NT>(p, ring, ahead);
                --to_issue;
            }
        }
        if (!ok) break;
        store_state8<D, NT>(p, st, row_at(p, gw, pair, inside ? 0 : 1));
        left -= cnt;
        at.off += cnt;
        if (at.off == at.units && left > 0) at.next_pair(p);
    }
    if (!ok && lane == 0) {
        // Let every copy this warp started land before the CTA exits.
        volatile int none = 0;
        for (uint32_t k = ring.used; k < ring.issued; ++k)
            mbar_wait(&ring.full[k % G::kStages], (k / G::kStages) & 1, &none, nullptr, p.timeout_ns);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- combine

// One CTA per query row, 1 to 8 warps: each warp joins every so-many-th of the row's
// partial states, a lane holding D / 32 columns, and the warps' sums meet in shared
// memory in warp order.
constexpr int kCombineWarps = 8;

template <int D, int NT>
__global__ void __launch_bounds__(32 * kCombineWarps) decode8_combine_kernel(const __grid_constant__ Decode8Params p, int most)
{
    constexpr int C = D / 32;  // columns per lane
    __shared__ float red_m[2][kCombineWarps], red_l[2][kCombineWarps], red_o[2][kCombineWarps][D];
    __shared__ Plan s_plan;
    __shared__ int s_before, s_T;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = (int)blockDim.x >> 5;
    const int pair = (int)(blockIdx.x / (unsigned)p.R), r = (int)(blockIdx.x % (unsigned)p.R);
    const int b = pair / p.Hkv, hk = pair % p.Hkv, tok = r % p.n;
    const float gate = p.gate[(long long)b * p.n + tok];
    const bool sel = takes_global(gate, *p.tau);
    if (warp == 0) {
        int T = 0, before = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const Plan pl = b0 + lane < p.B ? plan_of(p, b0 + lane) : Plan{0, 0, 0, 0};
            const int un = pl.units();
            T += (int)__reduce_add_sync(0xffffffffu, un) * p.Hkv;
            before += (int)__reduce_add_sync(0xffffffffu, b0 + lane < b ? un : 0) * p.Hkv;
            if (b0 + lane == b) s_plan = pl;
        }
        if (lane == 0) s_T = T, s_before = before;
    }
    __syncthreads();
    const Plan pl = s_plan;
    if (p.selected && hk == 0 && r < p.n && tid == 0) p.selected[(long long)b * p.n + r] = sel ? 1 : 0;
    uint16_t* out = p.out + ((long long)pair * p.R + r) * D;
    if (pl.len < p.n - tok) {  // the token lies before the sequence's start (or the length is invalid)
        for (int c = tid; c < D; c += (int)blockDim.x) out[c] = 0;
        return;
    }
    const Shares sh(s_T, most, least_units(NT));
    const int u0 = s_before + hk * pl.units();
    // slots of the states inside the window (kind 0) and, for a global token, before it (kind 1)
    const int w_in = sh.warp_of(u0 + pl.out), n_in = sh.warp_of(u0 + pl.units() - 1) - w_in + 1;
    const int w_out = sh.warp_of(u0), n_out = sel && pl.out ? sh.warp_of(u0 + pl.out - 1) - w_out + 1 : 0;
    const long long at[2] = {row_at(p, w_in, pair, 0) + r, row_at(p, w_out, pair, 1) + r};
    const int cnt[2] = {n_in, n_out};
    const float2* ml = part_ml(p);
    const float* po = part_o(p) + lane * C;
    const long long step = 2LL * p.R;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float m[2], l[2], o[2][C];
    #pragma unroll
    for (int k = 0; k < 2; ++k) {
        float mx = -INFINITY;
        for (int i = tid; i < cnt[k]; i += (int)blockDim.x) mx = fmaxf(mx, ml[at[k] + i * step].x);
        #pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        if (lane == 0) red_m[k][warp] = mx;
    }
    __syncthreads();
    #pragma unroll
    for (int k = 0; k < 2; ++k) {
        m[k] = -INFINITY;
        for (int w = 0; w < nw; ++w) m[k] = fmaxf(m[k], red_m[k][w]);
        l[k] = 0.f;
        #pragma unroll
        for (int c = 0; c < C; ++c) o[k][c] = 0.f;
        #pragma unroll 4
        for (int i = warp; i < cnt[k]; i += nw) {
            const long long row = at[k] + i * step;
            const float2 s = ml[row];
            float v[C];
            if (C == 4) {
                const float4 x = *reinterpret_cast<const float4*>(po + row * D);
                v[0] = x.x, v[1] = x.y, v[C - 2] = x.z, v[C - 1] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2*>(po + row * D);
                v[0] = x.x, v[1] = x.y;
            }
            const float f = s.x == -INFINITY ? 0.f : exp2f(s.x - m[k]);
            l[k] = fmaf(f, s.y, l[k]);
            #pragma unroll
            for (int c = 0; c < C; ++c) o[k][c] = fmaf(f, v[c], o[k][c]);
        }
    }
    if (nw > 1) {
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (lane == 0) red_l[k][warp] = l[k];
            #pragma unroll
            for (int c = 0; c < C; ++c) red_o[k][warp][lane * C + c] = o[k][c];
        }
        __syncthreads();
        if (warp > 0) return;
        #pragma unroll
        for (int k = 0; k < 2; ++k)
            for (int w = 1; w < nw; ++w) {
                l[k] += red_l[k][w];
                #pragma unroll
                for (int c = 0; c < C; ++c) o[k][c] += red_o[k][w][lane * C + c];
            }
    }
    float val[C];
    #pragma unroll
    for (int c = 0; c < C; ++c) val[c] = l[0] == 0.f ? 0.f : o[0][c] / l[0];
    if (sel) {
        const float M = fmaxf(m[0], m[1]);
        const float f0 = m[0] == -INFINITY ? 0.f : exp2f(m[0] - M), f1 = m[1] == -INFINITY ? 0.f : exp2f(m[1] - M);
        const float lt = fmaf(f0, l[0], f1 * l[1]), share = 1.f / (1.f + expf(-gate));
        #pragma unroll
        for (int c = 0; c < C; ++c) val[c] = fmaf(share, lt == 0.f ? 0.f : fmaf(f0, o[0][c], f1 * o[1][c]) / lt, val[c]);
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(out + lane * C);
    #pragma unroll
    for (int c = 0; c < C / 2; ++c) dst[c] = pack_bf16x2(val[2 * c], val[2 * c + 1]);
}

// CTAs of one wave on the current device (0 until asked), per kernel and device.
template <int TYPE, int D, int NT>
cudaError_t wave(int& grid)
{
    static std::atomic<int> known[64];
    using G = D8<D, NT>;
    auto kern = decode8_partial_kernel<TYPE, D, NT>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem)) != cudaSuccess) return e;
    grid = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (grid > 0) return cudaSuccess;
    int sms = 0, per_sm = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, G::kThreads, G::kSmem)) != cudaSuccess) return e;
    grid = sms * (per_sm > 0 ? per_sm : 1);
    if (grid > kDec8MaxWarps / G::kWarps) grid = kDec8MaxWarps / G::kWarps;
    if (dev < 64) known[dev].store(grid, std::memory_order_relaxed);
    return cudaSuccess;
}

template <int TYPE, int D, int NT>
cudaError_t launch_tdn(const Decode8Params& p, cudaStream_t stream)
{
    int grid = 0;
    cudaError_t e = wave<TYPE, D, NT>(grid);
    if (e != cudaSuccess) return e;
    decode8_partial_kernel<TYPE, D, NT><<<grid, D8<D, NT>::kThreads, D8<D, NT>::kSmem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // Warps per row: about four states for each, by the most that a row can have.
    const long long states = ((long long)grid * D8<D, NT>::kWarps) / ((long long)p.B * p.Hkv) + 2;
    const int warps = states <= 4 ? 1 : states <= 8 ? 2 : states <= 16 ? 4 : kCombineWarps;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hkv * p.R));
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode8_combine_kernel<D, NT>, p, grid * D8<D, NT>::kWarps);
}

template <int TYPE, int D>
cudaError_t launch_td(const Decode8Params& p, cudaStream_t stream)
{
    return p.R <= 8 ? launch_tdn<TYPE, D, 1>(p, stream)
                    : p.R <= 16 ? launch_tdn<TYPE, D, 2>(p, stream) : launch_tdn<TYPE, D, 4>(p, stream);
}

}  // namespace

size_t decode8_partials_bytes(int B, int Hkv, int R, int d)
{
    return (size_t)slots8((long long)B * Hkv) * 2 * R * (d + 2) * sizeof(float);
}

cudaError_t launch_decode8(const Decode8Params& p, int type, int d, cudaStream_t stream)
{
    if (type == kCacheE4M3) return d == 64 ? launch_td<kCacheE4M3, 64>(p, stream) : launch_td<kCacheE4M3, 128>(p, stream);
    return d == 64 ? launch_td<kCacheInt8, 64>(p, stream) : launch_td<kCacheInt8, 128>(p, stream);
}

}  // namespace logo
