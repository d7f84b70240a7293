// The 8-bit key/value cache: quantising new tokens as they are written, and
// reading rows back.
//
// A block of BLOCK tokens of one key/value head shares one fp32 scale (K and V
// apart).  With a = max(2^-100, largest finite |x| of the block's rows):
//     scale = a / Q,   code = RN(x Q / a),   value = code * scale,
// Q = 448 (e4m3) or 127 (int8), RN to the nearest value of the type, ties to even.
//
// Appending in pieces gives the same state as appending at once: the cache keeps
// the last two blocks' rows in bf16 (the tail; slot = block index mod 2), and an
// append that raises a block's maximum quantises the block's earlier rows again
// from there, never from codes.
//
// Correct rounding without a division per element.  x and a are bf16 (8-bit
// significands) and Q is 7 * 64 or 127, so x Q / a and a rounding border m (at
// most 8 significant bits) satisfy x Q = m a or differ relatively by at least
// 2^-16: both products are multiples of one power of two with at most 16
// significant bits (int8: 127 X < 2^15 against m A < 2^16).  The kernel forms
// x * fl(Q / a), off by a relative 2^-23 at most, and rounds that to 19 significant
// bits (error 2^-19) by Veltkamp's splitting (Dekker, "A floating-point technique for
// extending the available precision", 1971).  A quotient on a border is representable
// there and comes back exactly; any other stays on its side of every border.
//
// Both kernels are bound by HBM: 2 bytes read and 1 written per element (append),
// 1 read and 2 written (read back), each thread moving 16 elements at a time (32
// bytes of bf16, 16 bytes of codes).  A prompt of 32K tokens for 8 heads appended and
// read back: 66 us, 0.93 of the measured HBM bandwidth (e4m3; the append alone 29.8 us where
// its input is partly in L2, 2,048 tokens behind 4,096 for 8 sequences 15.8, one token for 64
// sequences 3.7, four 4.9).  The append was bound by the
// integer pipe (22 instructions an element in int8) until the rounding moved to the
// multiply-add pipe, whole numbers came from an addition instead of a conversion, and
// infinities and NaN got a copy of the loop of their own: 8 packed prompts in int8
// appended and read back 207 to 160 us.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "cache8.cuh"
#include "kernels.cuh"

namespace logo {

namespace {

// Threads of an append CTA: at most four vectors of 16 elements for each.
template <int D, int BLOCK>
constexpr int kA8ThreadsOf = D * BLOCK > 8192 ? 256 : 128;
// Threads per SM, by the registers of a thread: 64, for which all but the smallest blocks
// (64 x 64) spill 28 or 32 bytes.
constexpr int kA8Resident = 1024;
constexpr int kR8Threads = 128;

template <int TYPE>
struct Q8;
template <>
struct Q8<kCacheE4M3> {
    static constexpr float top = 448.f;
};
template <>
struct Q8<kCacheInt8> {
    static constexpr float top = 127.f;
};

struct alignas(32) Bf16x16 {
    uint32_t w[8];
};

__device__ __forceinline__ Bf16x16 load_bf16x16(const uint16_t* p)
{
    Bf16x16 v;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                   "=r"(v.w[7])
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void store_bf16x16(uint16_t* p, const Bf16x16& v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]),
                 "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
                 : "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x Q / a to 19 significant bits (see above): four operations of the multiply-add pipe,
// which has room where the integer pipe has none.
__device__ __forceinline__ float quotient(float x, float inv)
{
    const float y = __fmul_rn(x, inv), u = __fmul_rn(y, 33.f);
    return __fsub_rn(u, __fsub_rn(u, y));
}

// What stands for an input that is no finite number: +-inf saturates; NaN stays
// NaN in e4m3 and becomes 0 in int8.
template <int TYPE>
__device__ __forceinline__ float not_finite(float x)
{
    if (TYPE == kCacheE4M3) return x;
    return x != x ? 0.f : (x > 0.f ? 127.f : -127.f);
}

template <int TYPE>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    if (TYPE == kCacheE4M3) {
        uint16_t lo, hi;  // the first source goes to the upper byte
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return (uint32_t)lo | ((uint32_t)hi << 16);
    }
    // Adding 3 * 2^22 rounds to a whole number (ties to even) and leaves it, in two's
    // complement, in the low bits: |x| <= 127 needs the lowest byte only.
    constexpr float kWhole = 12582912.f;
    const uint32_t ab = __byte_perm(__float_as_uint(a + kWhole), __float_as_uint(b + kWhole), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(c + kWhole), __float_as_uint(d + kWhole), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
}

// ODD: some input of the block is no finite number.
template <int TYPE, bool ODD>
__device__ __forceinline__ uint32_t quant4(uint32_t w0, uint32_t w1, float inv)
{
    float x[4] = {bf16_lo(w0), bf16_hi(w0), bf16_lo(w1), bf16_hi(w1)};
    float y[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = quotient(x[i], inv);
        if (ODD && (__float_as_uint(x[i]) & 0x7f800000u) == 0x7f800000u) y[i] = not_finite<TYPE>(x[i]);
    }
    return pack4<TYPE>(y[0], y[1], y[2], y[3]);
}

// The rows that sequence b brings and where they lie in its head slab.  False (and
// reported) when the offsets or the target range are out of range; s is set all the same.
__device__ __forceinline__ bool span_of(const int32_t* cu, const int32_t* start, int b, int n_slab, int max_n,
                                        int Lmax, int& row0, int& n, int& s)
{
    row0 = 0;
    n = n_slab;
    s = start[b];
    if (cu) {
        row0 = cu[b];
        const long long e = cu[b + 1];
        if (row0 < 0 || e < row0 || e > n_slab || e - row0 > max_n) return false;
        n = (int)(e - row0);
    }
    return s >= 0 && (long long)s + n <= Lmax;
}

// One CTA per (sequence, key/value head, K or V, touched block).  All of the
// block's rows are held in registers (kept rows from the tail, new rows from the
// input), so the maximum and the codes need one pass over memory.  The earlier
// rows' codes are written again only when the block's scale changes.
template <int TYPE, int D, int BLOCK>
__global__ void __launch_bounds__(kA8ThreadsOf<D, BLOCK>, kA8Resident / kA8ThreadsOf<D, BLOCK>)
    append8_kernel(const __grid_constant__ Append8Params p)
{
    constexpr int kA8Threads = kA8ThreadsOf<D, BLOCK>;
    constexpr int kVecRow = D / 16;                           // 16-element vectors per row
    constexpr int kVec = BLOCK * kVecRow / kA8Threads;        // vectors per thread
    __shared__ uint32_t warp_max[kA8Threads / 32];
    const int Hkv = p.c.Hkv;
    long long it = blockIdx.x;
    const int j = (int)(it % p.nb);
    it /= p.nb;
    const int kv = (int)(it & 1);
    it >>= 1;
    const int hk = (int)(it % Hkv), b = (int)(it / Hkv);
    int row0, n, s;
    const bool ok = span_of(p.cu_seqlens, p.start, b, p.n, p.max_n, p.c.Lmax, row0, n, s);
    if (j == 0 && kv == 0 && hk == 0 && threadIdx.x == 0) {
        if (!ok) atomicOr(p.status, kStatusBadArgument);
        if (p.new_len) p.new_len[b] = ok ? s + n : s;
    }
    if (!ok) return;
    // (without new rows, what is left of the block is quantised without the rows taken back)
    const int first = s / BLOCK, blk = first + j, end = s + n, last = (end + BLOCK - 1) / BLOCK - 1;
    if (blk > last) return;
    const int base = blk * BLOCK;
    const int kept = j == 0 ? s - base : 0;
    const int rows = end - base < BLOCK ? end - base : BLOCK;
    const long long slab = (long long)b * Hkv + hk;
    // src points at the row that lands on position `base` (only rows >= kept exist)
    const uint16_t* head = p.src[kv] + (p.cu_seqlens ? (long long)hk * p.n + row0 : slab * p.n) * D;
    const uint16_t* src = head + (long long)(base - s) * D;
    uint16_t* tails = p.c.tail[kv] + slab * 2 * BLOCK * D;
    uint16_t* tail = tails + (blk & 1) * BLOCK * D;
    float* scale_at = p.c.scale[kv] + slab * p.c.nblk + blk;
    const float old_scale = kept > 0 ? *scale_at : 0.f;

    Bf16x16 x[kVec];
    uint32_t big = 0;  // largest magnitude, as the bits of a bf16 (both halves apart)
    #pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = threadIdx.x + i * kA8Threads, r = v / kVecRow, c = (v % kVecRow) * 16;
        if (r < rows) {
            x[i] = load_bf16x16(r < kept ? tail + r * D + c : src + r * D + c);
        } else {
            #pragma unroll
            for (int w = 0; w < 8; ++w) x[i].w[w] = 0u;
        }
    }
    #pragma unroll
    for (int i = 0; i < kVec; ++i)
        #pragma unroll
        for (int w = 0; w < 8; ++w) big = __vmaxu2(big, x[i].w[w] & 0x7fff7fffu);
    auto block_max = [&](uint32_t m2) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
        __syncthreads();
        uint32_t t = 0;
        #pragma unroll
        for (int w = 0; w < kA8Threads / 32; ++w) t = max(t, warp_max[w]);
        return t;
    };
    uint32_t top = block_max(big);
    const bool odd = top >= 0x7f80u;  // an infinity or NaN among the rows: the maximum is over the others
    if (odd) {
        big = 0;
        #pragma unroll
        for (int i = 0; i < kVec; ++i)
            #pragma unroll
            for (int w = 0; w < 8; ++w) {
                const uint32_t lo = x[i].w[w] & 0x7fffu, hi = (x[i].w[w] >> 16) & 0x7fffu;
                big = max(big, lo < 0x7f80u ? lo : 0u);
                big = max(big, hi < 0x7f80u ? hi : 0u);
            }
        __syncthreads();  // warp_max is read above
        top = block_max(big);
    }
    const float a = fmaxf(__uint_as_float(top << 16), kCache8Floor);
    const float scale = __fdiv_rn(a, Q8<TYPE>::top), inv = __fdiv_rn(Q8<TYPE>::top, a);
    // Every thread has read old_scale and its tail rows before the barrier in block_max.
    if (threadIdx.x == 0) *scale_at = scale;
    const int from = kept > 0 && __float_as_uint(old_scale) == __float_as_uint(scale) ? kept : 0;
    // Blocks `last - 1` and `last` go to the tail.  The first block's CTA writes the slot
    // that it reads its kept rows from, also for a later block of the same parity.
    const bool own_tail = blk >= last - 1 && (blk == first || ((blk - first) & 1));
    uint8_t* code = p.c.code[kv] + (slab * p.c.Lmax + base) * D;
    auto write_codes = [&](auto any_odd) {
        constexpr bool ODD = decltype(any_odd)::value;
        #pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = threadIdx.x + i * kA8Threads, r = v / kVecRow, c = (v % kVecRow) * 16;
            if (r < from || r >= rows) continue;
            uint4 o;
            o.x = quant4<TYPE, ODD>(x[i].w[0], x[i].w[1], inv);
            o.y = quant4<TYPE, ODD>(x[i].w[2], x[i].w[3], inv);
            o.z = quant4<TYPE, ODD>(x[i].w[4], x[i].w[5], inv);
            o.w = quant4<TYPE, ODD>(x[i].w[6], x[i].w[7], inv);
            *reinterpret_cast<uint4*>(code + r * D + c) = o;
        }
    };
    if (odd)
        write_codes(std::true_type{});
    else
        write_codes(std::false_type{});
    if (own_tail) {
        #pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = threadIdx.x + i * kA8Threads, r = v / kVecRow, c = (v % kVecRow) * 16;
            if (r >= kept && r < rows) store_bf16x16(tail + r * D + c, x[i]);
        }
    }
    if (j == 0) {
        const int other = ((last - first) & 1) ? last - 1 : last;  // the later block of this parity
        if (other > first) {
            const int obase = other * BLOCK, orows = end - obase < BLOCK ? end - obase : BLOCK;
            const uint16_t* osrc = head + (long long)(obase - s) * D;
            for (int v = threadIdx.x; v < orows * kVecRow; v += kA8Threads)
                store_bf16x16(tail + v * 16, load_bf16x16(osrc + v * 16));
        }
    }
}

// Four codes (one 32-bit word) as fp32.
template <int TYPE>
__device__ __forceinline__ void unpack4(uint32_t w, float (&x)[4])
{
    if (TYPE == kCacheE4M3) {
        uint32_t h0, h1;  // e4m3 to fp16 is exact
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(h0), "=r"(h1)
            : "r"(w));
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(x[0]), "=f"(x[1])
            : "r"(h0));
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(x[2]), "=f"(x[3])
            : "r"(h1));
    } else {
        #pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
    }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One CTA per (sequence, key/value head, K or V, kRead8Rows rows); every load of a
// thread is issued before its first use.
template <int TYPE, int D, int BLOCK>
__global__ void __launch_bounds__(kR8Threads) read8_kernel(const __grid_constant__ Read8Params p)
{
    constexpr int kVecRow = D / 16;
    constexpr int kVec = kRead8Rows * kVecRow / kR8Threads;
    const int Hkv = p.c.Hkv;
    long long it = blockIdx.x;
    const int j = (int)(it % p.nb);
    it /= p.nb;
    const int kv = (int)(it & 1);
    it >>= 1;
    const int hk = (int)(it % Hkv), b = (int)(it / Hkv);
    int row0, n, s;
    if (!span_of(p.cu_seqlens, p.start, b, p.n, p.max_n, p.c.Lmax, row0, n, s)) {
        if (j == 0 && kv == 0 && hk == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadArgument);
        return;
    }
    const int r0 = j * kRead8Rows, rows = n - r0 < kRead8Rows ? n - r0 : kRead8Rows;
    if (rows <= 0) return;
    const long long slab = (long long)b * Hkv + hk;
    const uint8_t* code = p.c.code[kv] + (slab * p.c.Lmax + s + r0) * D;
    const float* scales = p.c.scale[kv] + slab * p.c.nblk;
    uint16_t* dst = p.dst[kv] + ((p.cu_seqlens ? (long long)hk * p.n + row0 : slab * p.n) + r0) * D;
    uint4 x[kVec];
    float sc[kVec];
    #pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = threadIdx.x + i * kR8Threads, r = v / kVecRow;
        if (r >= rows) break;
        x[i] = *reinterpret_cast<const uint4*>(code + v * 16);
        sc[i] = scales[(s + r0 + r) / BLOCK];
    }
    #pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = threadIdx.x + i * kR8Threads, r = v / kVecRow;
        if (r >= rows) break;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        Bf16x16 o;
        #pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f[4];
            unpack4<TYPE>(w[q], f);
            o.w[2 * q] = bf16x2(f[0] * sc[i], f[1] * sc[i]);
            o.w[2 * q + 1] = bf16x2(f[2] * sc[i], f[3] * sc[i]);
        }
        store_bf16x16(dst + v * 16, o);
    }
}

template <int TYPE, int D>
cudaError_t append_td(const Append8Params& p, int block, unsigned grid, cudaStream_t stream)
{
    if (block == 64)
        append8_kernel<TYPE, D, 64><<<grid, kA8ThreadsOf<D, 64>, 0, stream>>>(p);
    else
        append8_kernel<TYPE, D, 128><<<grid, kA8ThreadsOf<D, 128>, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int TYPE, int D>
cudaError_t read_td(const Read8Params& p, int block, unsigned grid, cudaStream_t stream)
{
    if (block == 64)
        read8_kernel<TYPE, D, 64><<<grid, kR8Threads, 0, stream>>>(p);
    else
        read8_kernel<TYPE, D, 128><<<grid, kR8Threads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

// (the grids fit 31 bits: checked by the callers)
cudaError_t launch_append8(const Append8Params& p, int type, int d, int block, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((long long)p.c.B * p.c.Hkv * 2 * p.nb);
    if (type == kCacheE4M3)
        return d == 64 ? append_td<kCacheE4M3, 64>(p, block, grid, stream)
                       : append_td<kCacheE4M3, 128>(p, block, grid, stream);
    return d == 64 ? append_td<kCacheInt8, 64>(p, block, grid, stream)
                   : append_td<kCacheInt8, 128>(p, block, grid, stream);
}

cudaError_t launch_read8(const Read8Params& p, int type, int d, int block, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((long long)p.c.B * p.c.Hkv * 2 * p.nb);
    if (type == kCacheE4M3)
        return d == 64 ? read_td<kCacheE4M3, 64>(p, block, grid, stream)
                       : read_td<kCacheE4M3, 128>(p, block, grid, stream);
    return d == 64 ? read_td<kCacheInt8, 64>(p, block, grid, stream)
                   : read_td<kCacheInt8, 128>(p, block, grid, stream);
}

}  // namespace logo
