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
//   decode8_partial_kernel  one wave of persistent warps, 8 to an SM.  The work is a
//     list of units: for every (sequence, key/value head) the stages (8 KB of K and V: 32
//     positions, 64 at d = 64) before the window (only where a token is global), then the
//     stages that reach into it.
//     The list is cut into equal shares, one per warp, so every warp reads about the
//     same number of bytes whatever the lengths and gates are; the lengths are read on
//     the device.  A warp streams its stages through a private ring of 16 KB in shared
//     memory, filled by TMA (rows swizzled), tracked by one mbarrier per stage and kept
//     full from one sequence to the next.  Per stage:
//       S^T = K q^T   mma.sync m16n8k16, fp16 in, fp32 out: positions are the rows,
//                     the query rows the columns.  Codes become fp16 exactly.  The
//                     order of the head dimension inside a product is free, so a lane
//                     uses the four consecutive codes that ldmatrix gives it as they
//                     are, and q is stored in that order.
//       softmax       online, fp32; a maximum is taken only in stages that need one;
//       O^T += V^T P^T  V^T by ldmatrix.trans on pairs of codes: a word holds two
//                     head-dimension columns at two positions, and one byte permute
//                     sorts it into the fp16 pairs of two rows of V^T.  Each stage's
//                     product starts anew and joins O with the stage's V scale in
//                     fp32, so scales of any ratio meet only in 32 bits.
//     Positions outside the window and inside it go to separate partial states
//     (m, l, o; o as the mean of the values, so that no sum of states is larger than they
//     are): a position is read once, local attention is the inside state, global
//     attention both.  The warps of a CTA join their states in shared memory.
//   decode8_combine_kernel  one CTA per query row, placed while the first kernel runs where
//     that leaves registers (up to 8 rows; up to 16 at d = 64): joins the states of the CTAs
//     that held a share of the row's stages, in the order of the list;
//     o = local + sigmoid(g) * global, one rounding.
//
// mma.sync and not tcgen05: a stage of 8 KB takes an SM about 350 cycles to fetch and its
// 32 products a fraction of that, and codes need a conversion in registers, which an
// operand read from shared memory by tcgen05 would not see.
//
// Roundings: q is scaled by a power of two per row, so that its largest element lies
// in [2^14, 2^15), and rounded to fp16 (exact for elements down to 2^-28 of the
// largest).  P is held near 2^14 times itself in fp16: 11 bits, 3 more than bf16, with
// values down to 2^-38 of the largest kept.  The sum l uses the unrounded P.  The codes are
// exact: int8 codes as code + 128 in the products, less 128 times the other operand's sum, save
// two instructions of five for every four codes, but the roundings of sums that large stay
// where the codes are zero (16 rows: 77.4 against 80.5 us, four 61.1 against 61.9; d = 64, 32
// rows 78.2 against 74.7, where the correction costs more than it saves).
//
// Measured (d = 128, 32 query heads on 8, e4m3, window 4096; bytes that have to be read
// over the time, of the measured 6568 GB/s): 64 sequences of 32K, 13 global, 220 us
// (0.90; 195 to 216 where a call finds what the one before left in L2); one global sequence of 128K
// beside a local one 50.1 us (0.84); one of 32K 19.0 us (0.54); 16 of 8K to 32K with four
// drafted tokens each 58.4 us (0.69); two of 4K 8.9 us.  Once its first bytes are there (5 us:
// launch, lengths, the first 19 MB of all SMs' rings), a warp takes 2,650 to 3,000 cycles a
// stage, of which HBM alone asks 2,850; the kernel's end and the combine take 4 us.  From 9 rows
// on a warp's way through a stage (ldmatrix, conversion, products, softmax, movmatrix, products)
// is longer than its fetch, and with two warps a scheduler much of its latency shows: issue slots
// 38 to 46 % busy, tensor pipe 26 to 39 %, the largest stalls fixed latencies and the tensor pipe
// (370 MB for 4, 16, 24 and 32 rows a key/value head: 63, 74, 97, 118 us; int8 63, 80, 103, 131).
// A maximum for every stage in place of kPMargin: four drafts 64.6 us, 32 rows 185 us (with
// the six warps that its registers allowed), one token the same.
// Tried and left out: 64-position stages at d = 128 (four drafts 70 us), paired fp32
// instructions for the state (register moves: 72 us), chunks of the list's end fetched by a
// counter (64 sequences 220 us), rows finished by the last CTA of a pair instead of a second
// kernel (drafts 86 us), q fetched ahead (no change).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cache8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace logo {

namespace {

// P is held as 2^(s + nr): nr is kPBias less a maximum that the scores seen so far exceed by
// at most kPMargin, so that P stays below 2^16 and in fp16, and nearly every stage is done
// without finding its maximum across lanes or touching O.
// Scores are rounded to fp32 before nr is added, and nr is rounded down: however large they
// are, equal scores get equal P, and none above 2^(kPBias + kPMargin).  (The product in one
// multiply-add with nr would keep digits of it that nr has lost: infinite P at scores of 1e31.)
constexpr float kPBias = 14.f, kPMargin = 1.9f;
constexpr float kLargest = 3.402823466e38f;
constexpr float kEmpty = kLargest;  // nr while nothing was seen: scores above -kEmpty exceed it
constexpr int kWordsMax = 1024; // sequences whose length and gate decision a CTA keeps in shared memory

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= kLargest; }

template <int D, int NT>
struct D8 {
    static constexpr int kStage = dec8_stage(D);                  // positions of a stage
    static constexpr int kTile = kStage * D;                      // codes of K (or V) of one stage, bytes
    static constexpr int kStageBytes = 2 * kTile;                 // K then V
    static constexpr int kRingBytes = 16384;                      // of a warp; 128 KB in flight on an SM
    static constexpr int kStages = kRingBytes / kStageBytes;      // ring depth
    static constexpr int kQBytes = (D / 16) * NT * 32 * 8;        // q fragments of one warp
    static constexpr int kStateBytes = 8 * NT * (D + 2) * 4;      // partial state, written over the ring at the end
    static constexpr int kUsedBytes = kRingBytes + kQBytes > kStateBytes ? kRingBytes + kQBytes : kStateBytes;
    static constexpr int kWarpBytes = (kUsedBytes + 1023) / 1024 * 1024;
    // Two warps on every scheduler, and (up to 8 rows; 16 at d = 64) registers and shared memory
    // left for the combine kernel's CTAs (12 warps: they wait for the others to end, 10.4 -> 13.9
    // us for short contexts, 21.0 -> 25.0 us for one of 32K).
    static constexpr int kWarps = 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kSmem = kWarps * kWarpBytes + 1024;      // + alignment slack
    static constexpr int MT = kStage / 16;                        // 16-position tiles of a stage
    static_assert(kStages >= 2 && kSmem + 6 * 1024 <= 227 * 1024 && kWarps * 148 <= kDec8MaxWarps, "launch shape");
};

// ---------------------------------------------------------------- the list of units

__device__ __forceinline__ bool takes_global(float g, float tau) { return g > tau; }  // false for NaN

// A sequence's length with the sign bit set where one of its tokens is global; 0 for an
// empty sequence, kBadLength for one that the cache cannot hold.
constexpr uint32_t kGlobalBit = 0x80000000u, kBadLength = 0x40000001u;

__device__ __forceinline__ uint32_t word_from(const Decode8Params& p, int b)
{
    const int len = p.cache_len[b];
    const float tau = *p.tau;
    bool any = false;
    #pragma unroll 4
    for (int i = 0; i < p.n; ++i) any |= takes_global(p.gate[(long long)b * p.n + i], tau) && i >= p.n - len;
    if (len < 0 || len > p.Lmax) return kBadLength;
    return (uint32_t)len | (any ? kGlobalBit : 0u);
}

__device__ __noinline__ uint32_t word_far(const Decode8Params& p, int b) { return word_from(p, b); }

// Every thread of the CTA takes part; a barrier has to follow.
__device__ __forceinline__ void load_words(const Decode8Params& p, uint32_t* words)
{
    for (int b = threadIdx.x; b < p.B && b < kWordsMax; b += (int)blockDim.x) words[b] = word_from(p, b);
}
__device__ __forceinline__ uint32_t word_of(const Decode8Params& p, const uint32_t* words, int b)
{
    return b >= p.B ? 0u : b < kWordsMax ? words[b] : word_far(p, b);
}

// Units of one (sequence, key/value head): `out` stages before the window ([0, out),
// sequences with a global token only), then stages [in0, in1); they overlap in the stages
// that the first window edges of the n tokens cross.  Behind them lies one empty unit for
// either kind that there is: beginning a run and writing its state takes a warp about as
// long as a stage, and shares are equal in time where they count it (a batch of lengths 1
// to 16384 in int8: the slowest warp, with nine runs, took 102,000 cycles against 82,000
// for the others).
struct Plan {
    int len;  // 0 also for an invalid length
    int out, in0, in1;
    __device__ __forceinline__ Plan() : len(0), out(0), in0(0), in1(0) {}
    __device__ __forceinline__ Plan(const Decode8Params& p, uint32_t word) : Plan()
    {
        if (word == kBadLength) return;
        len = (int)(word & ~kGlobalBit);
        const int e0 = len - p.n - p.W + 1, e1 = len - p.W;  // window edges of the first and last token
        const int up = (1 << p.stage_log2) - 1;
        in0 = e0 > 0 ? e0 >> p.stage_log2 : 0;
        in1 = (len + up) >> p.stage_log2;
        out = (word & kGlobalBit) && e1 > 0 ? (e1 + up) >> p.stage_log2 : 0;
    }
    __device__ __forceinline__ int stages() const { return out + in1 - in0; }
    __device__ __forceinline__ int units() const { return stages() + (len > 0 ? 1 : 0) + (out > 0 ? 1 : 0); }
};

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

// T units cut into N shares, at most `most`, none of them empty: the first `rest` shares
// have one unit more than the others.  T fits 32 bits: a unit is at least 4 KB of
// cache, read at most twice.
struct Shares {
    int N, each, rest;
    __device__ __forceinline__ Shares(int T, int most)
    {
        N = T < most ? T : most;
        each = T < most ? 1 : (int)((unsigned)T / (unsigned)most);  // T below `most`: shares of one unit
        rest = T < most ? 0 : T - each * N;
    }
    __device__ __forceinline__ int first(int w) const { return w * each + (w < rest ? w : rest); }
    __device__ __forceinline__ int of(int u) const  // the share that unit u belongs to
    {
        const bool big = u < rest * (each + 1);
        const unsigned n = big ? each + 1 : each, x = big ? u : u - rest;
        return (int)(x / n);  // behind the big shares: rest + (u - rest (each + 1)) / each
    }
};

// The list is cut into one share per CTA, and that into one per warp.  A run is the
// stages of one pair (sequence, key/value head) and one kind (0: inside the window, 1:
// before it).  A warp's last run goes on in the next warp, as a rule: the CTA joins those
// states and writes one for the run's first warp in the CTA.  A run that ends inside a
// warp's share is written by that warp alone.
//
// Behind the workspace's header: for every sequence the units ahead of it, then the whole
// list's (written by CTA 0, read by the combine kernel where the batch is large).
__host__ __device__ inline long long prefix8(long long B) { return (B + 1 + 63) / 64 * 64; }
__device__ __forceinline__ int* prefix_of(const Decode8Params& p)
{
    return reinterpret_cast<int*>(p.part) - prefix8(p.B);
}
// Sequences up to which a CTA of the combine kernel adds up the lengths itself, while the
// partial kernel runs, and above which it reads the sums that CTA 0 of that wrote.  Either way
// for 512 positions of 2 heads, 4 rows (us): 2 sequences 7.4 and 7.8, 32 8.8 and 9.3, 64 11.5 and
// 11.7, 96 13.5 and 13.6, 128 15.4 and 15.3, 256 24.5 and 21.5, 1,024 97 and 68; with 24 rows
// at d = 64: 64 17.9 and 17.8, 128 27.1 and 24.9.
constexpr int kScanMax = 64;

// Partial states lie in slots of R rows and two kinds, (m, l) and o apart.  Slot (warp of
// the grid + pair) is unique, since along the list either the warp or the pair moves on.
__host__ __device__ inline long long slots8(long long pairs) { return kDec8MaxWarps + pairs; }
__device__ __forceinline__ long long row_at(const Decode8Params& p, int gw, int pair, int kind)
{
    return (((long long)gw + pair) * 2 + kind) * p.R;
}
__device__ __forceinline__ float2* part_ml(const Decode8Params& p) { return reinterpret_cast<float2*>(p.part); }
__device__ __forceinline__ float* part_o(const Decode8Params& p)
{
    return p.part + slots8((long long)p.B * p.Hkv) * 2 * p.R * 2;
}

// ---------------------------------------------------------------- fragments

template <int OFF>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFF));
}

template <int OFF>
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFF));
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

// The same from zero (which costs no register).
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// O is held as kOScale times sum P v (the V scale takes it along): with P's 2^14 the smallest
// values (scales of 2^-109) keep their digits.
constexpr float kOScale = 0x1p-17f;
// A V scale up to kVsMax adds less than 2^96 to O with each position (P < 2^16, codes < 2^9), so
// that 2^30 positions stay below 2^126.  The first larger one of a run takes a factor of kShrink
// off O and off every V scale from there on, which is enough for any finite scale.
constexpr float kVsMax = 0x1p88f, kShrink = 0x1p-40f;

// Codes as fp16 pairs, exact.  int8: a code + 128 as the low byte of fp16's 1024 is 1152 + code.
__device__ __forceinline__ uint32_t less_1152(uint32_t x)
{
    uint32_t y;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x64806480u));
    return y;
}

template <int TYPE>
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)  // bytes 0, 1 and 2, 3
{
    if (TYPE == kCacheE4M3) {
        asm("{\n\t.reg .b16 x, y;\n\t"
            "mov.b32 {x, y}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, x;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t u = w ^ 0x80808080u;
        lo = less_1152(__byte_perm(u, 0x64646464u, 0x4140));
        hi = less_1152(__byte_perm(u, 0x64646464u, 0x4342));
    }
}

// A word of ldmatrix.trans holds two positions' codes of columns 2g and 2g + 1: bytes
// (pos 0: 2g, 2g + 1; pos 1: 2g, 2g + 1).  As fp16 pairs over the positions: column 2g,
// column 2g + 1.
template <int TYPE>
__device__ __forceinline__ void to_f16_pairs(uint32_t w, uint32_t& even, uint32_t& odd)
{
    if (TYPE == kCacheE4M3) {
        to_f16<TYPE>(__byte_perm(w, 0u, 0x3120), even, odd);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        even = less_1152(__byte_perm(u, 0x64646464u, 0x4240));
        odd = less_1152(__byte_perm(u, 0x64646464u, 0x4341));
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

__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* status,
                                       unsigned long long limit_ns)
{
    return mbar_wait(bar, parity, abort_flag, status, limit_ns);
}

// Softmax state of the warp's query rows.  Lane (g, t) = (lane / 4, lane % 4) has
// columns 8 nt + 2t + c (c = 0, 1): their nr (shared by the 8 lanes of the same t; the
// state that is written has m = -nr), a share of their sums, and of O^T the rows
// 16 u + 2g + h at o[u][nt][2h + c].
template <int D, int NT>
struct State8 {
    float nr[NT][2], l[NT][2];
    float o[D / 16][NT][4];
    float fx;  // 1, or kShrink
    __device__ __forceinline__ void init()
    {
        fx = 1.f;
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) nr[nt][0] = nr[nt][1] = kEmpty, l[nt][0] = l[nt][1] = 0.f;
        #pragma unroll
        for (int u = 0; u < D / 16; ++u)
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) o[u][nt][0] = o[u][nt][1] = o[u][nt][2] = o[u][nt][3] = 0.f;
    }
};

__device__ __forceinline__ float fast_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / x for a sum of weights x >= 0; 0 where there are none.
__device__ __forceinline__ float share_of(float x) { return x == 0.f ? 0.f : fast_rcp(x); }

__device__ __forceinline__ void store_if(bool yes, void* at, float a, float b)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t@q st.v2.f32 [%1], {%2, %3};\n\t}" ::"r"((int)yes), "l"(at),
                 "f"(a), "f"(b)
                 : "memory");
}

// The state's rows to (m, l) at ml[r] and o at o[r * D], in shared or global memory; o is written as
// the mean sum P v / sum P, which is no larger than the values, however many they are.  Predicated
// stores and no branches: this code runs once or twice in a launch, and every branch of it
// would wait for its instructions.
template <int TYPE, int D, int NT>
__device__ __forceinline__ void store_state8(State8<D, NT>& st, int R, float2* ml, float* o)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    #pragma unroll
    for (int off = 4; off < 32; off <<= 1)
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            #pragma unroll
            for (int c = 0; c < 2; ++c) st.l[nt][c] += __shfl_xor_sync(0xffffffffu, st.l[nt][c], off);
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = 8 * nt + 2 * t + c;
            const float f = share_of(st.l[nt][c] * (kOScale * st.fx));
            store_if(r < R && g == 0, ml + r, -st.nr[nt][c], st.l[nt][c]);
            float* row = o + r * D + 2 * g;
            #pragma unroll
            for (int u = 0; u < D / 16; ++u)
                store_if(r < R, row + 16 * u, st.o[u][nt][c] * f, st.o[u][nt][2 + c] * f);
        }
}

// Joins the states of warps first .. last of the CTA, held in their shared memory (`at`: the
// first warp's; o, then (m, l)), row by row: this warp takes every so-many-th row.
template <int D, int NT>
__device__ __forceinline__ void join_states(const Decode8Params& p, const uint8_t* at, int size, int rank, long long row)
{
    constexpr int C = D / 32, kWarps = D8<D, NT>::kWarps;  // lanes 0 .. kWarps - 1 hold a warp's (m, l) each
    const int lane = threadIdx.x & 31;
    for (int r = rank; r < p.R; r += size) {
        auto ml = [&](int i) {
            return reinterpret_cast<const float2*>(at + (long long)i * D8<D, NT>::kWarpBytes + 8 * NT * D * 4)[r];
        };
        const float2 mine = lane < size ? ml(lane) : make_float2(-INFINITY, 0.f);
        float m = mine.x;
        #pragma unroll
        for (int off = kWarps / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float w = mine.y * fast_exp2(mine.x - m);
        float l = w, o[C];
        #pragma unroll
        for (int off = kWarps / 2; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        const float f_mine = w * share_of(l);
        #pragma unroll
        for (int c = 0; c < C; ++c) o[c] = 0.f;
        #pragma unroll 4
        for (int i = 0; i < size; ++i) {
            const float f = __shfl_sync(0xffffffffu, f_mine, i);
            const float* src = reinterpret_cast<const float*>(at + (long long)i * D8<D, NT>::kWarpBytes) + r * D + lane;
            #pragma unroll
            for (int c = 0; c < C; ++c) o[c] = fmaf(f, src[32 * c], o[c]);
        }
        if (lane == 0) part_ml(p)[row + r] = make_float2(m, l);
        float* dst = part_o(p) + (row + r) * D + lane;
        #pragma unroll
        for (int c = 0; c < C; ++c) dst[32 * c] = o[c];
    }
}

// Where in the list a warp's copies are: unit `off` of key/value head hk of sequence b.
struct Cursor {
    int b, hk, off;
    Plan pl;
    // To the next pair's first unit.
    __device__ __forceinline__ void next_pair(const Decode8Params& p, const uint32_t* words)
    {
        off = 0;
        if (++hk < p.Hkv) return;
        hk = 0;
        do {
            if (++b >= p.B) return;
            pl = Plan(p, word_of(p, words, b));
        } while (pl.len == 0);
    }
};

// The next unit's keys and values into the ring (all lanes keep count, lane 0 copies), and
// beside them what the warp has to know of the stage: the run (2 pair + kind), the stage's
// index in the sequence and the sequence's length.
template <int D, int NT>
__device__ __forceinline__ void issue_unit(const Decode8Params& p, Ring8& ring, int4* units, Cursor& at)
{
    using G = D8<D, NT>;
    const bool inside = at.off >= at.pl.out;
    const int stage = inside ? at.off - at.pl.out + at.pl.in0 : at.off, pair = at.b * p.Hkv + at.hk;
    const uint32_t s = ring.issued % G::kStages;
    if ((threadIdx.x & 31) == 0) {
        uint8_t* dst = reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(ring.base + s * G::kStageBytes));
        // the warp's reads of this stage come before the copy engine's writes
        if (ring.issued >= (uint32_t)G::kStages) fence_proxy_async_smem();
        mbar_arrive_expect_tx(&ring.full[s], G::kStageBytes);
        tma_load_3d(dst, &p.tm_k, &ring.full[s], 0, stage * G::kStage, pair, policy_evict_first());
        tma_load_3d(dst + G::kTile, &p.tm_v, &ring.full[s], 0, stage * G::kStage, pair, policy_evict_first());
        units[s] = make_int4(2 * pair + (inside ? 0 : 1), stage, at.pl.len, 0);
    }
    ++ring.issued;
    ++at.off;
}

// Per-lane constants of the (sequence, key/value head) at hand.
template <int NT>
struct Rows8 {
    float qf[NT][2];  // scale * log2(e) / (the power of two in the row's fp16 q)
    int tok[NT][2];   // the column's token
};

// q of one (sequence, key/value head) to fp16 in shared memory, in fragment order: lane
// (g, t) of unit kk, tile nt holds row 8 nt + g, elements 16 kk + 4t .. + 3.
template <int TYPE, int D, int NT>
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
        ex = ex > 126 ? 126 : ex;
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
            rw.qf[nt][c] = p.scale_log2 * __uint_as_float((uint32_t)(127 - e2) << 23);
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
    for (int k = lane; k < dec8_stage(D) * D / 16; k += 32) {
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
    for (int r = 0; r < dec8_stage(D); ++r) {
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

// One stage: scores, softmax step, products.  `masked`: some column sees it in part, or the
// V scale is above kVsMax or not finite.
template <int TYPE, int D, int NT>
__device__ __forceinline__ void do_stage(State8<D, NT>& st, const Rows8<NT>& rw, const uint2* qs, uint32_t tileK,
                                         float ks, float vs, bool masked, int pos0, int lo0, int hi0, int n)
{
    using G = D8<D, NT>;
    constexpr int MT = G::MT;
    constexpr int H = MT / 2;  // ldmatrix of V^T per 16 columns: 32 positions each
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const uint32_t tileV = tileK + G::kTile;
    if (masked) {
        if (mask_values<TYPE, D>(tileV, pos0, lo0, hi0, n) && TYPE == kCacheE4M3)
            place_nan<D, NT>(tileV, pos0, lo0, hi0, n, rw, st);
        if (finite(vs)) {
            if (fabsf(vs) > kVsMax) {
                vs *= kShrink;
                st.fx *= kShrink;
                #pragma unroll
                for (int u = 0; u < D / 16; ++u)
                    #pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) st.o[u][nt][e] *= kShrink;
            }
        } else {
            // NaN for the columns that see the stage; the others' products are zero, which times
            // such a scale would be NaN too.
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                #pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (lo0 + rw.tok[nt][c] < pos0 + G::kStage && hi0 + rw.tok[nt][c] >= pos0)
                        st.l[nt][c] = __int_as_float(0x7fffffff);
            vs = 0.f;
        }
    }
    // S^T = K q^T: rows = positions 16 mt + g (+ 8), columns = query rows.  ldmatrix: lane's row
    // lane mod 16 of the 16, 16-byte unit 2 kk + lane / 16; the swizzle turns into an exclusive or.
    float sc[MT][NT][4];
    const uint32_t kat = swz<D>(tileK, lane & 15, lane >> 4);
    #pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
        uint2 b0[NT], b1[NT];
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            b0[nt] = qs[((2 * kk) * NT + nt) * 32 + lane];
            b1[nt] = qs[((2 * kk + 1) * NT + nt) * 32 + lane];
        }
        // every product of a step before the first that continues one
        uint32_t x[MT][4], y[MT][4];
        #pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t w[4];
            switch (mt) {
                case 0: ldsm4<0>(kat ^ (kk << 5), w); break;
                case 1: ldsm4<16 * D>(kat ^ (kk << 5), w); break;
                case 2: ldsm4<32 * D>(kat ^ (kk << 5), w); break;
                default: ldsm4<48 * D>(kat ^ (kk << 5), w); break;
            }
            #pragma unroll
            for (int q = 0; q < 4; ++q) to_f16<TYPE>(w[q], x[mt][q], y[mt][q]);
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (kk == 0)
                    mma_f16_zero(sc[mt][nt], x[mt][0], x[mt][1], y[mt][0], y[mt][1], b0[nt].x, b0[nt].y);
                else
                    mma_f16(sc[mt][nt], x[mt][0], x[mt][1], y[mt][0], y[mt][1], b0[nt].x, b0[nt].y);
            }
        }
        #pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_f16(sc[mt][nt], x[mt][2], x[mt][3], y[mt][2], y[mt][3], b1[nt].x, b1[nt].y);
    }
    // Online softmax, in units of log2.
    uint32_t pb[MT][NT][2];
    float mx[NT][2];
    bool over = false;
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float f = ks * rw.qf[nt][c];
            #pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                #pragma unroll
                for (int h = 0; h < 2; ++h) sc[mt][nt][2 * h + c] = __fmul_rn(sc[mt][nt][2 * h + c], f);
            if (masked) {
                const int lo = lo0 + rw.tok[nt][c] - pos0 - g, hi = hi0 + rw.tok[nt][c] - pos0 - g;
                #pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    #pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (16 * mt + 8 * h < lo || 16 * mt + 8 * h > hi) sc[mt][nt][2 * h + c] = -INFINITY;
            }
            mx[nt][c] = fmaxf(sc[0][nt][c], sc[0][nt][2 + c]);
            #pragma unroll
            for (int mt = 1; mt < MT; ++mt) mx[nt][c] = fmax3(mx[nt][c], sc[mt][nt][c], sc[mt][nt][2 + c]);
            over |= __fadd_rn(mx[nt][c], st.nr[nt][c]) > kPBias + kPMargin;
        }
    if (__any_sync(0xffffffffu, over)) {
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float al[2];
            #pragma unroll
            for (int c = 0; c < 2; ++c) {
                #pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    mx[nt][c] = fmaxf(mx[nt][c], __shfl_xor_sync(0xffffffffu, mx[nt][c], off));
                const float nr = fminf(st.nr[nt][c], __fsub_rd(kPBias, mx[nt][c]));
                al[c] = fast_exp2(nr - st.nr[nt][c]);  // 0 while nothing was seen
                st.nr[nt][c] = nr;
                st.l[nt][c] *= al[c];
            }
            #pragma unroll
            for (int u = 0; u < D / 16; ++u)
                #pragma unroll
                for (int e = 0; e < 4; ++e) st.o[u][nt][e] *= al[e & 1];
        }
    }
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[2];
                #pragma unroll
                for (int c = 0; c < 2; ++c) {
                    x[c] = fast_exp2(__fadd_rn(sc[mt][nt][2 * h + c], st.nr[nt][c]));
                    st.l[nt][c] += x[c];
                }
                // P^T fragment: the score fragment's 8x8 quarter transposed in registers
                pb[mt][nt][h] = movm(pack_f16x2(x[0], x[1]));
            }
    // O^T += (V^T P^T) vs
    vs *= kOScale;
    const uint32_t vat = swz<D>(tileV, lane, 0);
    #pragma unroll
    for (int u = 0; u < D / 16; ++u) {
        uint32_t ev[H][4], od[H][4];
        #pragma unroll
        for (int h = 0; h < H; ++h) {
            uint32_t w[4];
            if (h == 0)
                ldsm4t<0>(vat ^ (u << 4), w);
            else
                ldsm4t<32 * D>(vat ^ (u << 4), w);
            #pragma unroll
            for (int i = 0; i < 4; ++i) to_f16_pairs<TYPE>(w[i], ev[h][i], od[h][i]);
        }
        float acc[NT][4];
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            mma_f16_zero(acc[nt], ev[0][0], od[0][0], ev[0][1], od[0][1], pb[0][nt][0], pb[0][nt][1]);
        #pragma unroll
        for (int mt = 1; mt < MT; ++mt)
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_f16(acc[nt], ev[mt / 2][2 * (mt & 1)], od[mt / 2][2 * (mt & 1)], ev[mt / 2][2 * (mt & 1) + 1],
                        od[mt / 2][2 * (mt & 1) + 1], pb[mt][nt][0], pb[mt][nt][1]);
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            #pragma unroll
            for (int e = 0; e < 4; ++e) st.o[u][nt][e] = fmaf(acc[nt][e], vs, st.o[u][nt][e]);
    }
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(D8<D, NT>::kThreads, 1) decode8_partial_kernel(const __grid_constant__ Decode8Params p)
{
    using G = D8<D, NT>;
    extern __shared__ uint8_t dsmem8[];
    __shared__ uint64_t full_bars[G::kWarps][G::kStages];
    __shared__ uint32_t words[kWordsMax];
    __shared__ int abort_word;
    __shared__ int4 unit_info[G::kWarps][G::kStages];
    __shared__ int last_run[G::kWarps];  // 2 pair + kind of each warp's last run, -1: none
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
    // Let the combine kernel's CTAs be placed; they wait for this grid's end before they read.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t was = *reinterpret_cast<volatile uint32_t*>(p.status);
    if (lane == 0) {
        for (int s = 0; s < G::kStages; ++s) mbar_init(&full_bars[warp][s], 1);
        fence_barrier_init();
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    load_words(p, words);
    if (threadIdx.x == 0) abort_word = (was & kStatusTimeout) ? 1 : 0;
    __syncthreads();
    volatile int* abort_flag = &abort_word;
    // The whole list's length (every warp for itself).
    int T = 0, incl = 0;
    bool bad = false;
    Plan mine;
    for (int b = lane; b - lane < p.B; b += 32) {
        const uint32_t w = word_of(p, words, b);
        bad |= w == kBadLength;
        mine = Plan(p, w);
        incl = warp_scan(mine.units()) * p.Hkv;
        if (p.B > kScanMax && blockIdx.x == 0 && warp == G::kWarps - 1 && b < p.B)
            prefix_of(p)[b] = T + incl - mine.units() * p.Hkv;
        T += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (p.B > kScanMax && blockIdx.x == 0 && threadIdx.x == 0) prefix_of(p)[p.B] = T;
    // An earlier call's wait ran out: nothing is attended to, but the combine kernel, which
    // places its reads by them, has this call's sums.
    if (*abort_flag) return;
    if (bad && blockIdx.x == 0 && warp == 0) atomicOr(p.status, kStatusBadArgument);
    const Shares ctas(T, (int)gridDim.x);
    const int cta = (int)blockIdx.x;
    if (cta >= ctas.N) return;
    const int u_cta = ctas.first(cta);
    const Shares sh(ctas.first(cta + 1) - u_cta, G::kWarps);
    const int gw = cta * G::kWarps + warp;
    int to_issue = warp < sh.N ? sh.first(warp + 1) - sh.first(warp) : 0;
    Cursor at{};
    if (to_issue > 0) {
        int before = u_cta + sh.first(warp);  // units ahead of the share, less those of the sequences passed
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            if (p.B > 32) {  // else they are still here
                mine = Plan(p, word_of(p, words, b0 + lane));
                incl = warp_scan(mine.units()) * p.Hkv;
            }
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
            const int units = at.pl.units();
            before -= __shfl_sync(0xffffffffu, incl, src) - units * p.Hkv;
            at.hk = (int)((unsigned)before / (unsigned)units);
            at.off = before - at.hk * units;
            break;
        }
    }
    const uint32_t base = ((smem_u32(dsmem8) + 1023u) & ~1023u) + warp * G::kWarpBytes;
    uint2* qs = reinterpret_cast<uint2*>(__cvta_shared_to_generic(base + G::kRingBytes));
    Ring8 ring{base, full_bars[warp], 0, 0};
    int run = -1, lo0 = 0, hi0 = 0, first = 0, last = 0;
    float ks32 = 0.f, vs32 = 0.f;  // scales of stages first .. first + 31, one per lane
    bool ok = true, new_q = false;
    Rows8<NT> rw;
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = 8 * nt + 2 * t + c;
            rw.tok[nt][c] = r - p.n * (int)((r + 0.5f) / (float)p.n);  // r mod n, both at most 32
        }
    State8<D, NT> st;
    st.init();
    for (;;) {
        while (to_issue > 0 && ring.issued - ring.used < (uint32_t)G::kStages) {
            if (at.off >= at.pl.stages()) {  // the empty units at a pair's end
                to_issue -= at.pl.units() - at.off;
                at.next_pair(p, words);
                continue;
            }
            issue_unit<D, NT>(p, ring, unit_info[warp], at);
            --to_issue;
        }
        __syncwarp();
        const uint32_t s = ring.used % G::kStages;
        const bool done = ring.used == ring.issued;
        const int4 unit = done ? make_int4(-1, 0, 0, 0) : unit_info[warp][s];
        if (unit.x != run || done) {
            if (done) break;       // the share's last state stays in registers
            if (run >= 0) {        // a run ends inside the share: its state goes to its slot
                const long long row = row_at(p, gw, run >> 1, run & 1);
                store_state8<TYPE, D, NT>(st, p.R, part_ml(p) + row, part_o(p) + row * D);
            }
            // token i sees [lo0 + i, hi0 + i]: its window, or what lies before it (lo0 then at
            // most 0 for every token)
            const bool inside = !(unit.x & 1);
            lo0 = inside ? unit.z - p.n - p.W + 1 : -kDec8MaxRows;
            hi0 = unit.z - p.n - (inside ? 0 : p.W);
            first = -64;
            last = (unit.z - 1) / G::kStage;
            new_q = run < 0 || (unit.x ^ run) > 1;
            run = unit.x;
            st.init();
        }
        if (unit.y - first >= 32) {
            first = unit.y;
            const int blk = (first + lane < last ? first + lane : last) / p.block_units;
            ks32 = p.k_scale[(long long)(run >> 1) * p.nblk + blk];
            vs32 = p.v_scale[(long long)(run >> 1) * p.nblk + blk];
        }
        if (new_q) stage_q<TYPE, D, NT>(p, run >> 1, qs, rw);  // while the scales are on their way
        new_q = false;
        const float ks = __shfl_sync(0xffffffffu, ks32, unit.y - first);
        const float vs = __shfl_sync(0xffffffffu, vs32, unit.y - first) * st.fx;
        const uint32_t parity = (ring.used / G::kStages) & 1;
        ok = mbar_try_wait(&ring.full[s], parity) || wait_long(&ring.full[s], parity, abort_flag, p.status, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int pos0 = unit.y * G::kStage;
        const bool masked = pos0 < lo0 + p.n - 1 || pos0 + G::kStage - 1 > hi0 || !(fabsf(vs) <= kVsMax);
        do_stage<TYPE, D, NT>(st, rw, qs, ring.base + s * G::kStageBytes, ks, vs, masked, pos0, lo0, hi0, p.n);
        ++ring.used;
        __syncwarp();  // every lane is done with the stage
    }
    if (!ok) {
        run = -1;
        if (lane == 0) {  // let every copy this warp started land before the CTA exits
            volatile int none = 0;
            for (uint32_t k = ring.used; k < ring.issued; ++k)
                wait_long(&ring.full[k % G::kStages], (k / G::kStages) & 1, &none, nullptr, p.timeout_ns);
        }
        __syncwarp();
    }
    // The warps' last runs, joined where neighbours share one.
    if (lane == 0) last_run[warp] = run;
    __syncthreads();
    int lo = warp, hi = warp;
    if (run >= 0) {
        while (lo > 0 && last_run[lo - 1] == run) --lo;
        while (hi + 1 < G::kWarps && last_run[hi + 1] == run) ++hi;
        const long long row = row_at(p, gw, run >> 1, run & 1);
        float* own = reinterpret_cast<float*>(__cvta_shared_to_generic(base));  // over the ring
        store_state8<TYPE, D, NT>(st, p.R, lo == hi ? part_ml(p) + row : reinterpret_cast<float2*>(own + 8 * NT * D),
                            lo == hi ? part_o(p) + row * D : own);
    }
    __syncthreads();
    if (lo < hi)
        join_states<D, NT>(p, reinterpret_cast<const uint8_t*>(__cvta_shared_to_generic(base)) - (warp - lo) * G::kWarpBytes,
                           hi - lo + 1, warp - lo, row_at(p, cta * G::kWarps + lo, run >> 1, run & 1));
}

// ---------------------------------------------------------------- combine

// One CTA per query row, 1 to 4 warps: each warp joins every so-many-th of the row's
// partial states, a lane holding D / 32 columns, and the warps' sums meet in shared
// memory in warp order.
constexpr int kCombineWarps = 4;

template <int D, int NT>
__global__ void __launch_bounds__(32 * kCombineWarps) decode8_combine_kernel(const __grid_constant__ Decode8Params p, int grid)
{
    constexpr int C = D / 32;  // columns per lane
    constexpr int kWarps = D8<D, NT>::kWarps;
    __shared__ float red_m[2][kCombineWarps], red_l[2][kCombineWarps];
    __shared__ alignas(16) float red_o[2][kCombineWarps][D];
    __shared__ int s_before[kCombineWarps], s_T[kCombineWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = (int)blockDim.x >> 5;
    const int pair = (int)(blockIdx.x / (unsigned)p.R), r = (int)(blockIdx.x % (unsigned)p.R);
    const int b = pair / p.Hkv, hk = pair % p.Hkv, tok = r % p.n;
    const float gate = p.gate[(long long)b * p.n + tok];
    const bool sel = takes_global(gate, *p.tau);
    int T = 0, before = 0;
    if (p.B <= kScanMax) {
        for (int i = tid; i < p.B; i += (int)blockDim.x) {
            const int un = Plan(p, word_from(p, i)).units() * p.Hkv;
            T += un;
            if (i < b) before += un;
        }
        T = (int)__reduce_add_sync(0xffffffffu, T);
        before = (int)__reduce_add_sync(0xffffffffu, before);
        if (lane == 0) s_T[warp] = T, s_before[warp] = before;
        __syncthreads();
        T = before = 0;
        for (int w = 0; w < nw; ++w) T += s_T[w], before += s_before[w];
    }
    const Plan pl(p, word_from(p, b));
    if (p.selected && hk == 0 && r < p.n && tid == 0) p.selected[(long long)b * p.n + r] = sel ? 1 : 0;
    uint16_t* out = p.out + ((long long)pair * p.R + r) * D;
    if (pl.len < p.n - tok) {  // the token lies before the sequence's start, or the length is invalid
        asm volatile("griddepcontrol.wait;" ::: "memory");  // no CTA ends ahead of the partial kernel
        for (int c = tid; c < D; c += (int)blockDim.x) out[c] = 0;
        return;
    }
    if (p.B > kScanMax) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        before = __ldcg(prefix_of(p) + b);
        T = __ldcg(prefix_of(p) + p.B);
    }
    // Where the row's states lie: for each CTA that the run reaches into, the slot of the run's
    // first warp there; and the run's last warp's own where its share goes on behind the run.
    const Shares ctas(T, grid);
    const int u0 = before + hk * pl.units();
    const int from[2] = {u0 + pl.out, u0}, to[2] = {u0 + pl.stages(), u0 + (sel ? pl.out : 0)};
    int cnt[2], extra[2];
    long long row0[2], row1[2], row_x[2];
    #pragma unroll
    for (int k = 0; k < 2; ++k) {
        cnt[k] = extra[k] = 0;
        row0[k] = row1[k] = row_x[k] = 0;
        if (from[k] >= to[k]) continue;
        const int c0 = ctas.of(from[k]), c1 = ctas.of(to[k] - 1);
        const Shares s0(ctas.first(c0 + 1) - ctas.first(c0), kWarps);
        const Shares s1(ctas.first(c1 + 1) - ctas.first(c1), kWarps);
        const int v0 = s0.of(from[k] - ctas.first(c0)), v1 = s1.of(to[k] - 1 - ctas.first(c1));
        cnt[k] = c1 - c0 + 1;
        row0[k] = row_at(p, c0 * kWarps + v0, pair, k) + r;      // in the first CTA
        row1[k] = row_at(p, (c0 + 1) * kWarps, pair, k) + r;     // in the next, kWarps slots from one to the next
        // (the empty units behind a pair's last run are no other run)
        const int behind = k == 0 ? u0 + pl.units() : to[k];
        extra[k] = s1.first(v1 + 1) > behind - ctas.first(c1) && v1 != (c1 == c0 ? v0 : 0);
        row_x[k] = row_at(p, c1 * kWarps + v1, pair, k) + r;
    }
    const float2* ml = part_ml(p);
    const float* po = part_o(p) + lane * C;
    const long long step = 2LL * p.R * kWarps;
    auto row_of = [&](int k, int i) {
        return i == 0 ? row0[k] : i < cnt[k] ? row1[k] + (i - 1) * step : row_x[k];
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Each warp joins its states kJoin at a time, all of their loads in flight together; then
    // warp 0 joins the warps'.  o is a mean of values throughout, l the sum of the weights.
    constexpr int kJoin = 8;
    float m[2], l[2], o[2][C];
    #pragma unroll
    for (int k = 0; k < 2; ++k) {
        m[k] = -INFINITY, l[k] = 0.f;
        #pragma unroll
        for (int c = 0; c < C; ++c) o[k][c] = 0.f;
    }
    auto load = [&](const float* at, float (&v)[C]) {
        if (C == 4) {
            const float4 x = *reinterpret_cast<const float4*>(at);
            v[0] = x.x, v[1] = x.y, v[C - 2] = x.z, v[C - 1] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2*>(at);
            v[0] = x.x, v[1] = x.y;
        }
    };
    // weight of a state with maximum x among those with maximum y >= x
    auto weight = [](float x, float y) { return x == -INFINITY ? 0.f : fast_exp2(x - y); };
    const int all = cnt[0] + extra[0] + cnt[1] + extra[1];
    #pragma unroll 1
    for (int i0 = warp; i0 < all; i0 += kJoin * nw) {
        float2 s[kJoin];
        float v[kJoin][C];
        bool outside[kJoin];
        float mx[2] = {m[0], m[1]};
        #pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const int i = i0 + j * nw;
            outside[j] = i >= cnt[0] + extra[0];
            s[j] = make_float2(-INFINITY, 0.f);
            #pragma unroll
            for (int c = 0; c < C; ++c) v[j][c] = 0.f;
            if (i < all) {
                const long long row = outside[j] ? row_of(1, i - cnt[0] - extra[0]) : row_of(0, i);
                s[j] = ml[row];
                load(po + row * D, v[j]);
            }
        }
        #pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            mx[0] = fmaxf(mx[0], outside[j] ? -INFINITY : s[j].x);
            mx[1] = fmaxf(mx[1], outside[j] ? s[j].x : -INFINITY);
        }
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float was = weight(m[k], mx[k]) * l[k];
            float w[kJoin];
            m[k] = mx[k];
            l[k] = was;
            #pragma unroll
            for (int j = 0; j < kJoin; ++j) {
                w[j] = weight(s[j].x, mx[k]) * s[j].y;
                l[k] = outside[j] == (k == 1) ? l[k] + w[j] : l[k];
            }
            const float f = share_of(l[k]);
            #pragma unroll
            for (int c = 0; c < C; ++c) o[k][c] *= was * f;
            #pragma unroll
            for (int j = 0; j < kJoin; ++j) {
                // (a weight of zero does not hide a state that is NaN)
                const bool here = outside[j] == (k == 1);
                #pragma unroll
                for (int c = 0; c < C; ++c) o[k][c] = here ? fmaf(w[j] * f, v[j][c], o[k][c]) : o[k][c];
            }
        }
    }
    if (nw > 1) {
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (lane == 0) red_m[k][warp] = m[k], red_l[k][warp] = l[k];
            #pragma unroll
            for (int c = 0; c < C; ++c) red_o[k][warp][lane * C + c] = o[k][c];
        }
        __syncthreads();
        if (warp > 0) return;
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
            float x[kCombineWarps], w[kCombineWarps], mx = m[k];
            #pragma unroll
            for (int i = 0; i < kCombineWarps; ++i) {
                x[i] = i < nw ? red_m[k][i] : -INFINITY;
                w[i] = i < nw ? red_l[k][i] : 0.f;
                mx = fmaxf(mx, x[i]);
            }
            m[k] = mx;
            l[k] = 0.f;
            #pragma unroll
            for (int i = 0; i < kCombineWarps; ++i) l[k] += w[i] *= weight(x[i], mx);
            const float f = share_of(l[k]);
            #pragma unroll
            for (int c = 0; c < C; ++c) o[k][c] *= w[0] * f;
            #pragma unroll
            for (int i = 1; i < kCombineWarps; ++i) {
                if (i >= nw) break;
                float v[C];
                load(&red_o[k][i][lane * C], v);
                #pragma unroll
                for (int c = 0; c < C; ++c) o[k][c] = fmaf(w[i] * f, v[c], o[k][c]);
            }
        }
    }
    float val[C];
    #pragma unroll
    for (int c = 0; c < C; ++c) val[c] = o[0][c];
    if (sel) {
        const float M = fmaxf(m[0], m[1]);
        const float w0 = weight(m[0], M) * l[0], w1 = weight(m[1], M) * l[1];
        const float f = share_of(w0 + w1), share = 1.f / (1.f + expf(-gate));
        #pragma unroll
        for (int c = 0; c < C; ++c) val[c] = fmaf(share, fmaf(w0 * f, o[0][c], w1 * f * o[1][c]), val[c]);
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
    const long long states = grid / ((long long)p.B * p.Hkv) + 2;
    const int warps = states <= 4 ? 1 : states <= 8 ? 2 : kCombineWarps;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hkv * p.R));
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode8_combine_kernel<D, NT>, p, grid);
}

// Products, exponentials and O's registers go by eights of rows, so each count of eights has
// its kernel (24 rows in that of 32, 371 MB: e4m3 119 against 100 us, int8 132 against 105;
// d = 64, 186 MB: 74 against 58, 76 against 63).
template <int TYPE, int D>
cudaError_t launch_td(const Decode8Params& p, cudaStream_t stream)
{
    return p.R <= 8 ? launch_tdn<TYPE, D, 1>(p, stream)
           : p.R <= 16 ? launch_tdn<TYPE, D, 2>(p, stream)
           : p.R <= 24 ? launch_tdn<TYPE, D, 3>(p, stream) : launch_tdn<TYPE, D, 4>(p, stream);
}

}  // namespace

size_t decode8_partials_bytes(int B, int Hkv, int R, int d)
{
    return (size_t)(prefix8(B) + slots8((long long)B * Hkv) * 2 * R * (d + 2)) * sizeof(float);
}

cudaError_t launch_decode8(const Decode8Params& params, int type, int d, cudaStream_t stream)
{
    Decode8Params p = params;
    p.part += prefix8(p.B);
    p.stage_log2 = d == 64 ? 6 : 5;
    p.block_units = p.block >> p.stage_log2;
    if (type == kCacheE4M3) return d == 64 ? launch_td<kCacheE4M3, 64>(p, stream) : launch_td<kCacheE4M3, 128>(p, stream);
    return d == 64 ? launch_td<kCacheInt8, 64>(p, stream) : launch_td<kCacheInt8, 128>(p, stream);
}

}  // namespace logo

