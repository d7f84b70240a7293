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
//     Warp w takes units [w T / N, (w+1) T / N) of the T, so every warp reads the same
//     number of bytes whatever the lengths and gates are; the lengths are read on the
//     device.  A warp streams its stages through a private ring in shared memory,
//     filled by TMA (rows swizzled) and tracked by one mbarrier per stage.  Per stage:
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

__device__ __forceinline__ Plan plan_of(const Decode8Params& p, int b)
{
    Plan pl{0, 0, 0, 0};
    const int len = p.cache_len[b];
    if (len <= 0 || len > p.Lmax) return pl;
    bool any = false;
    const float tau = *p.tau;
    for (int i = p.n > len ? p.n - len : 0; i < p.n; ++i) any |= takes_global(p.gate[(long long)b * p.n + i], tau);
    // window edges of the first and last token (32-bit: W <= Lmax and n <= 32)
    const long long e0 = (long long)len - p.n - p.W + 1, e1 = (long long)len - p.W;
    pl.len = len;
    pl.in0 = e0 > 0 ? (int)(e0 / kDec8Stage) : 0;
    pl.in1 = (len + kDec8Stage - 1) / kDec8Stage;
    pl.out = any && e1 > 0 ? (int)((e1 + kDec8Stage - 1) / kDec8Stage) : 0;
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

// Warps that share T units: at most `most`, each with at least two units.
__device__ __forceinline__ long long warps_for(long long T, long long most)
{
    const long long w = (T + 1) / 2;
    return w < most ? w : most;
}
__device__ __forceinline__ long long first_unit(long long w, long long T, long long N) { return w * T / N; }
__device__ __forceinline__ long long warp_of(long long u, long long T, long long N) { return ((u + 1) * N - 1) / T; }

// Partial states: slot (warp + pair) is unique, since along the list either the warp
// or the pair (sequence, key/value head) moves on from one share to the next.
template <int D>
__device__ __forceinline__ float* slot_of(const Decode8Params& p, long long warp, long long pair, int kind)
{
    return p.part + (((warp + pair) * 2 + kind) * p.R) * (D + 2);
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
__device__ __forceinline__ void store_state8(const State8<D, NT>& st, int R, float* dst)
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
            if (r >= R) continue;
            float* row = dst + (long long)r * (D + 2);
            if (g == 0) *reinterpret_cast<float2*>(row) = make_float2(st.m[nt][c], l);
            #pragma unroll
            for (int u = 0; u < D / 16; ++u)
                *reinterpret_cast<float2*>(row + 2 + 16 * u + 2 * g) =
                    make_float2(st.o[u][nt][c], st.o[u][nt][2 + c]);
        }
    }
}

template <int D, int NT>
__device__ __forceinline__ void issue_stage(const Decode8Params& p, Ring8& ring, int stage, int slab)
{
    using G = D8<D, NT>;
    const uint32_t s = ring.issued % G::kStages;
    uint8_t* dst = reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(ring.base + s * G::kStageBytes));
    fence_proxy_async_smem();  // the warp's ldmatrix reads of this stage come before the copy engine's writes
    mbar_arrive_expect_tx(&ring.full[s], G::kStageBytes);
    tma_load_3d(dst, &p.tm_k, &ring.full[s], 0, stage * kDec8Stage, slab, policy_evict_first());
    tma_load_3d(dst + G::kTile, &p.tm_v, &ring.full[s], 0, stage * kDec8Stage, slab, policy_evict_first());
}

// O^T += V^T P^T over one softmax step (16 MT positions from smem row `row0`), times
// the V scale.  MASKED: codes at positions whose bit in `vm` is clear count as zero
// (the cache may hold anything there), and only columns where `cols` says so are
// added to.
template <int TYPE, int D, int NT, bool MASKED>
__device__ __forceinline__ void add_pv(State8<D, NT>& st, uint32_t tileV, int row0, const uint32_t (&pb)[D8<D, NT>::MT][NT][2],
                                       const float (&al)[NT][2], float vs, const uint32_t* vm, const bool (*cols)[2])
{
    constexpr int MT = D8<D, NT>::MT;
    const int lane = threadIdx.x & 31;
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
            for (int i = 0; i < 4; ++i) {
                if (MASKED) w[i] &= vm[4 * h + i];
                // bytes (pos 0: column 2g, 2g+1; pos 1: 2g, 2g+1) -> (2g: pos 0, 1; 2g+1: pos 0, 1)
                to_f16<TYPE>(__byte_perm(w[i], 0u, 0x3120), ev[i], od[i]);
            }
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
            for (int e = 0; e < 4; ++e) {
                const float was = st.o[u][nt][e] * al[nt][e & 1];
                if (!MASKED || cols[nt][e & 1]) st.o[u][nt][e] = fmaf(acc[nt][e], vs, was);
            }
    }
}

// Per-lane constants of the (sequence, key/value head) at hand.
template <int NT>
struct Rows8 {
    float qf[NT][2];  // scale * log2(e) / (the power of two in the row's fp16 q)
    int tok[NT][2];   // the column's token
};

// Stages [a, e) of slab `slab`.  A column of token i sees positions [lo0 + i, hi0 + i]
// when `inside`, else [0, hi0 + i]; hi may be negative (nothing seen).  `len` positions
// of the cache are held.  Returns false when a wait ran out (the CTA aborts).
template <int TYPE, int D, int NT>
__device__ __forceinline__ bool run_stages(const Decode8Params& p, Ring8& ring, State8<D, NT>& st, const Rows8<NT>& rw,
                                           const uint2* qs, int a, int e, int slab, bool inside, int lo0, int hi0, int len,
                                           volatile int* abort_flag)
{
    using G = D8<D, NT>;
    constexpr int MT = G::MT, kSteps = 4 / MT;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int cnt = e - a;
    if (lane == 0)
        for (int i = 0; i < cnt && i < G::kStages; ++i) {
            issue_stage<D, NT>(p, ring, a + i, slab);
            ++ring.issued;
        }
    ring.issued = ring.used + (cnt < G::kStages ? cnt : G::kStages);
    // Scales of 32 stages at a time, one stage per lane.
    const float* ksp = p.k_scale + (long long)slab * p.nblk;
    const float* vsp = p.v_scale + (long long)slab * p.nblk;
    float ks32 = 0.f, vs32 = 0.f;
    const int kr = (lane & 7) + 8 * ((lane >> 3) & 1), ku = lane >> 4;  // ldmatrix roles: row, 16-byte unit
    const int lo_max = inside ? max(lo0 + p.n - 1, 0) : 0;              // every column sees [lo_max, hi0]
    for (int i = 0; i < cnt; ++i) {
        if ((i & 31) == 0) {
            const int blk = (a + i + lane) / p.block_units;
            ks32 = i + lane < cnt ? ksp[blk] : 0.f;
            vs32 = i + lane < cnt ? vsp[blk] : 0.f;
        }
        const float ks = __shfl_sync(0xffffffffu, ks32, i & 31), vs = __shfl_sync(0xffffffffu, vs32, i & 31);
        const uint32_t s = ring.used % G::kStages;
        const bool ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[s], (ring.used / G::kStages) & 1, abort_flag, p.status,
                                                          p.timeout_ns));
        if (!ok) return false;
        const uint32_t tileK = ring.base + s * G::kStageBytes, tileV = tileK + G::kTile;
        const int pos0 = (a + i) * kDec8Stage;
        const bool masked = pos0 < lo_max || pos0 + kDec8Stage - 1 > hi0;
        #pragma unroll
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
            #pragma unroll
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
                    float mx = -INFINITY;
                    #pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        #pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float x = sc[mt][nt][2 * h + c] * f;
                            if (masked) {
                                const int pos = pos0 + row0 + 16 * mt + 8 * h + g, i0 = rw.tok[nt][c];
                                if ((inside && pos < lo0 + i0) || pos > hi0 + i0) x = -INFINITY;
                            }
                            sc[mt][nt][2 * h + c] = x;
                            mx = fmaxf(mx, x);
                        }
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
            if (!masked) {
                add_pv<TYPE, D, NT, false>(st, tileV, row0, pb, al, vs, nullptr, nullptr);
                continue;
            }
            // A stage that some column sees in part.  Codes that no column sees are taken as
            // zero.  With several tokens a code may be NaN at a position that only some of
            // them see: then one product per token, over that token's positions.
            const int first = inside ? lo0 : 0, last = hi0 + p.n - 1;
            uint32_t vm[2 * MT];
            bool cols[NT][2];
            auto set_mask = [&](int lo, int hi) {
                #pragma unroll
                for (int k = 0; k < 2 * MT; ++k) {
                    const int q = pos0 + row0 + 8 * k + 2 * t;
                    vm[k] = (q >= lo && q <= hi ? 0x0000ffffu : 0u) | (q + 1 >= lo && q + 1 <= hi ? 0xffff0000u : 0u);
                }
            };
            bool nan = false;
            if (TYPE == kCacheE4M3 && p.n > 1) {
                for (int k = lane; k < 16 * MT * D / 16; k += 32) {
                    const uint4 w = *reinterpret_cast<const uint4*>(
                        __cvta_shared_to_generic(tileV + row0 * D + 16 * k));
                    nan |= (__vcmpeq4(w.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(w.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                            __vcmpeq4(w.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(w.w & 0x7f7f7f7fu, 0x7f7f7f7fu)) != 0u;
                }
                nan = __any_sync(0xffffffffu, nan);
            }
            const int passes = nan ? p.n : 1;
            for (int i0 = 0; i0 < passes; ++i0) {
                if (passes == 1)
                    set_mask(first, last < len - 1 ? last : len - 1);
                else
                    set_mask(inside ? lo0 + i0 : 0, hi0 + i0);
                #pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    #pragma unroll
                    for (int c = 0; c < 2; ++c) cols[nt][c] = passes == 1 || rw.tok[nt][c] == i0;
                add_pv<TYPE, D, NT, true>(st, tileV, row0, pb, al, vs, vm, cols);
            }
        }
        ++ring.used;
        __syncwarp();
        if (i + G::kStages < cnt) {
            if (lane == 0) issue_stage<D, NT>(p, ring, a + i + G::kStages, slab);
            ++ring.issued;
        }
    }
    return true;
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(D8<D, NT>::kThreads, 1) decode8_partial_kernel(const __grid_constant__ Decode8Params p)
{
    using G = D8<D, NT>;
    extern __shared__ uint8_t dsmem8[];
    __shared__ uint64_t full_bars[G::kWarps][G::kStages];
    __shared__ int abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // Let the combine kernel's CTAs be placed; they wait for this grid's end before they read.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) abort_word = (*reinterpret_cast<volatile uint32_t*>(p.status) & kStatusTimeout) ? 1 : 0;
    if (lane == 0) {
        for (int s = 0; s < G::kStages; ++s) mbar_init(&full_bars[warp][s], 1);
        fence_barrier_init();
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    __syncthreads();
    volatile int* abort_flag = &abort_word;
    if (*abort_flag) return;
    const uint32_t base = ((smem_u32(dsmem8) + 1023u) & ~1023u) + warp * G::kWarpBytes;
    uint2* qs = reinterpret_cast<uint2*>(__cvta_shared_to_generic(base + G::kRingBytes));
    Ring8 ring{base, full_bars[warp], 0, 0};

    // The whole list's length, then this warp's share of it.
    long long T = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        int u = 0;
        if (b < p.B) {
            const int len = p.cache_len[b];
            if ((len < 0 || len > p.Lmax) && blockIdx.x == 0 && warp == 0) atomicOr(p.status, kStatusBadArgument);
            u = plan_of(p, b).units();
        }
        T += (long long)__reduce_add_sync(0xffffffffu, u) * p.Hkv;
    }
    if (T == 0) return;
    const long long N = warps_for(T, (long long)gridDim.x * G::kWarps);
    const long long gw = (long long)warp * gridDim.x + blockIdx.x;  // few warps: one per SM first
    if (gw >= N) return;
    long long u = first_unit(gw, T, N);
    const long long u_end = first_unit(gw + 1, T, N);
    bool ok = true;
    long long before = 0;  // units of the sequences before this group of 32
    for (int b0 = 0; b0 < p.B && u < u_end && ok; b0 += 32) {
        const Plan mine = b0 + lane < p.B ? plan_of(p, b0 + lane) : Plan{0, 0, 0, 0};
        const int incl = warp_scan(mine.units());
        const long long group = (long long)__shfl_sync(0xffffffffu, incl, 31) * p.Hkv;
        while (u < u_end && u < before + group && ok) {
            const unsigned past = __ballot_sync(0xffffffffu, before + (long long)incl * p.Hkv > u);
            const int src = __ffs(past) - 1, b = b0 + src;
            Plan pl;
            pl.len = __shfl_sync(0xffffffffu, mine.len, src);
            pl.out = __shfl_sync(0xffffffffu, mine.out, src);
            pl.in0 = __shfl_sync(0xffffffffu, mine.in0, src);
            pl.in1 = __shfl_sync(0xffffffffu, mine.in1, src);
            const int units = pl.units();
            const long long at = u - before - (long long)(__shfl_sync(0xffffffffu, incl, src) - units) * p.Hkv;
            const int hk = (int)(at / units), off = (int)(at % units);
            const int stop = u_end - u < units - off ? off + (int)(u_end - u) : units;  // share [off, stop)
            u += stop - off;
            // q in fp16 fragment order: lane (g, t) of unit kk, tile nt holds row 8 nt + g, elements
            // 16 kk + 4t .. + 3
            const long long pair = (long long)b * p.Hkv + hk;
            const uint16_t* q = p.q + pair * p.R * D;
            Rows8<NT> rw;
            __syncwarp();
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = 8 * nt + g;
                uint2 w[D / 16];
                uint32_t big = 0;
                #pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    w[kk] = r < p.R ? *reinterpret_cast<const uint2*>(q + (long long)r * D + 16 * kk + 4 * t)
                                    : make_uint2(0u, 0u);
                    big = __vmaxu2(big, __vmaxu2(w[kk].x & 0x7fff7fffu, w[kk].y & 0x7fff7fffu));
                }
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
            const int slab = (int)pair;
            State8<D, NT> st;
            if (off < pl.out) {  // before the window: token i sees [0, len - n - W + i]
                st.init();
                ok = run_stages<TYPE, D, NT>(p, ring, st, rw, qs, off, stop < pl.out ? stop : pl.out, slab, false, 0,
                                             pl.len - p.n - p.W, pl.len, abort_flag);
                if (!ok) break;
                store_state8<D, NT>(st, p.R, slot_of<D>(p, gw, pair, 1));
            }
            if (stop > pl.out) {  // the window: token i sees [len - n - W + 1 + i, len - n + i]
                const int a = (off > pl.out ? off - pl.out : 0) + pl.in0;
                st.init();
                ok = run_stages<TYPE, D, NT>(p, ring, st, rw, qs, a, stop - pl.out + pl.in0, slab, true,
                                             pl.len - p.n - p.W + 1, pl.len - p.n, pl.len, abort_flag);
                if (!ok) break;
                store_state8<D, NT>(st, p.R, slot_of<D>(p, gw, pair, 0));
            }
        }
        before += group;
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

template <int D>
__global__ void __launch_bounds__(D) decode8_combine_kernel(const __grid_constant__ Decode8Params p, long long most)
{
    __shared__ float red[D / 32];
    __shared__ Plan s_plan;
    __shared__ long long s_before, s_T;
    const int col = threadIdx.x, lane = col & 31;
    const long long pair = blockIdx.x / p.R;
    const int r = (int)(blockIdx.x % p.R);
    const int b = (int)(pair / p.Hkv), hk = (int)(pair % p.Hkv), tok = r % p.n;
    if (col < 32) {
        long long T = 0, before = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const Plan pl = b0 + lane < p.B ? plan_of(p, b0 + lane) : Plan{0, 0, 0, 0};
            const int un = pl.units();
            T += (long long)__reduce_add_sync(0xffffffffu, un) * p.Hkv;
            before += (long long)__reduce_add_sync(0xffffffffu, b0 + lane < b ? un : 0) * p.Hkv;
            if (b0 + lane == b) s_plan = pl;
        }
        if (lane == 0) s_T = T, s_before = before;
    }
    __syncthreads();
    const Plan pl = s_plan;
    const long long T = s_T;
    const float gate = p.gate[(long long)b * p.n + tok];
    const bool sel = takes_global(gate, *p.tau);
    if (p.selected && hk == 0 && r < p.n && col == 0) p.selected[(long long)b * p.n + r] = sel ? 1 : 0;
    uint16_t* out = p.out + (pair * p.R + r) * D;
    if (pl.len < p.n - tok) {  // the token lies before the sequence's start (or the length is invalid)
        out[col] = 0;
        return;
    }
    const long long N = warps_for(T, most);
    const long long u0 = s_before + (long long)hk * pl.units();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (m, l, o) joined over the warps w0 .. w1 that hold stages of the given kind
    auto join = [&](int kind, long long a, long long e, float& m, float& l, float& o) {
        m = -INFINITY, l = 0.f, o = 0.f;
        if (a >= e) return;
        const long long w0 = warp_of(u0 + a, T, N), w1 = warp_of(u0 + e - 1, T, N);
        const float* st = slot_of<D>(p, w0, pair, kind) + (long long)r * (D + 2);
        const long long step = 2LL * p.R * (D + 2);
        const int cnt = (int)(w1 - w0 + 1);
        float mx = -INFINITY;
        for (int k = col; k < cnt; k += D) mx = fmaxf(mx, st[k * step]);
        #pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        __syncthreads();
        if (lane == 0) red[col >> 5] = mx;
        __syncthreads();
        #pragma unroll
        for (int w = 0; w < D / 32; ++w) m = fmaxf(m, red[w]);
        #pragma unroll 8
        for (int k = 0; k < cnt; ++k) {
            const float* s = st + k * step;
            const float f = s[0] == -INFINITY ? 0.f : exp2f(s[0] - m);
            l = fmaf(f, s[1], l);
            o = fmaf(f, s[2 + col], o);
        }
    };
    float m, l, o;
    join(0, pl.out, pl.units(), m, l, o);
    float val = l == 0.f ? 0.f : o / l;
    if (sel) {
        float m1, l1, o1;
        join(1, 0, pl.out, m1, l1, o1);
        const float M = fmaxf(m, m1);
        const float f0 = m == -INFINITY ? 0.f : exp2f(m - M), f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - M);
        const float lt = fmaf(f0, l, f1 * l1), ot = fmaf(f0, o, f1 * o1);
        val = fmaf(1.f / (1.f + expf(-gate)), lt == 0.f ? 0.f : ot / lt, val);
    }
    const __nv_bfloat16 y = __float2bfloat16_rn(val);
    out[col] = *reinterpret_cast<const uint16_t*>(&y);
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
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hkv * p.R));
    cfg.blockDim = dim3(D);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode8_combine_kernel<D>, p, (long long)grid * D8<D, NT>::kWarps);
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
    return ((size_t)kDec8MaxWarps + (size_t)B * Hkv) * 2 * R * (d + 2) * sizeof(float);
}

cudaError_t launch_decode8(const Decode8Params& p, int type, int d, cudaStream_t stream)
{
    if (type == kCacheE4M3) return d == 64 ? launch_td<kCacheE4M3, 64>(p, stream) : launch_td<kCacheE4M3, 128>(p, stream);
    return d == 64 ? launch_td<kCacheInt8, 64>(p, stream) : launch_td<kCacheInt8, 128>(p, stream);
}

}  // namespace logo
