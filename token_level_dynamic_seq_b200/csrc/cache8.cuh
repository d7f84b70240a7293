// Launch interface between the C ABI (api.cu) and the kernels of the 8-bit key/value cache.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace logo {

enum Cache8Type : int { kCacheE4M3 = 0, kCacheInt8 = 1 };

// A block's largest magnitude counts as at least 2^-100, so that its scale and the
// reciprocal of its scale are normal fp32 numbers whatever the block holds.
constexpr float kCache8Floor = 7.888609052210118e-31f;

// One cache: codes [B, Hkv, Lmax, d], scales [B, Hkv, nblk], tails [B, Hkv, 2, block, d];
// index 0 holds the keys, index 1 the values.
struct Cache8View {
    uint8_t* code[2];
    float* scale[2];
    uint16_t* tail[2];
    int B, Hkv, Lmax, nblk;
};

struct Append8Params {
    Cache8View c;
    const uint16_t* src[2];     // new rows: [B, Hkv, n, d], or [Hkv, T, d] packed
    const int32_t* start;       // [B]
    const int32_t* cu_seqlens;  // nullptr: fixed length
    int32_t* new_len;           // [B] or nullptr
    uint32_t* status;
    int n;      // rows of a head slab: n (fixed) or T (packed)
    int max_n;  // longest sequence
    int nb;     // blocks that one sequence's new rows can touch, at most
};

struct Read8Params {
    Cache8View c;
    uint16_t* dst[2];           // [B, Hkv, n, d], or [Hkv, T, d] packed
    const int32_t* start;       // [B]
    const int32_t* cu_seqlens;  // nullptr: fixed length
    uint32_t* status;
    int n, max_n;
    int nb;  // blocks of kRead8Rows rows of the longest sequence
};
constexpr int kRead8Rows = 64;  // rows per CTA of the read

cudaError_t launch_append8(const Append8Params& p, int type, int d, int block, cudaStream_t stream);
cudaError_t launch_read8(const Read8Params& p, int type, int d, int block, cudaStream_t stream);

// Decode over the cache (decode8.cu).
// Cache positions per staged unit: 4 KB of K and as much of V.  Every scale block is a
// multiple of it.
__host__ __device__ constexpr int dec8_stage(int d) { return 4096 / d; }
constexpr int kDec8MaxRows = 32;      // query rows (heads of a group x new tokens) of one key/value head
constexpr int kDec8MaxWarps = 1184;   // warps that a launch spreads the work over, at most (148 SMs x 8)

struct alignas(64) Decode8Params {
    CUtensorMap tm_k, tm_v;     // codes as [B*Hkv][Lmax][d] bytes, box d x dec8_stage(d) x 1, swizzled rows
    const uint16_t* q;          // [B, Hq, n, d]
    const float *k_scale, *v_scale;
    const int32_t* cache_len;   // [B], the new tokens included
    const float* gate;          // [B, n]
    const float* tau;           // one threshold (device)
    uint16_t* out;              // [B, Hq, n, d]
    int32_t* selected;          // [B, n] or nullptr
    float* part;                // the workspace behind its header
    uint32_t* status;
    int B, Hkv, R, n, Lmax, W, nblk;
    int block;                  // positions per scale block
    int stage_log2, block_units;  // set at the launch: positions per stage, stages per scale block
    float scale_log2;
    unsigned long long timeout_ns;
};
size_t decode8_partials_bytes(int B, int Hkv, int R, int d);
cudaError_t launch_decode8(const Decode8Params& p, int type, int d, cudaStream_t stream);

}  // namespace logo
