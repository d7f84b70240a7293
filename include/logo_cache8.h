/*
 * logo_cache8.h -- the 8-bit key/value cache of the library: quantising new
 * tokens into it, reading rows back, and the decode step over it.
 *
 * The decode step reads every cache byte it needs once and does little else
 * ("Learning When to Attend", "Empirical Validation and System Optimization":
 * the gains carry over to generation, whose global reads are memory-bound), so
 * a cache of half the bytes takes about half the time and half the memory.
 *
 * Conventions are those of logo.h: the caller owns every buffer, nothing is
 * allocated or synchronised, every call is asynchronous on `stream` on the
 * current device, argument errors are reported before anything is launched and
 * device-side ones through the workspace's status word (logo_check).
 */
#ifndef LOGO_CACHE8_H_
#define LOGO_CACHE8_H_

#include "logo.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LOGO_CACHE_E4M3 = 0, /* 8-bit floats, 4 exponent and 3 fraction bits, largest value Q = 448 */
    LOGO_CACHE_INT8 = 1  /* whole numbers -127 .. 127, Q = 127 */
} logo_cache_type;

/*
 * One layer's cache.  A block of `block` tokens (64 or 128) of one key/value
 * head has one fp32 scale, keys and values apart.  With a = max(2^-100, largest
 * finite |x| of the block's rows):
 *   scale = a / Q (fp32), code = x * Q / a rounded to the nearest value of the
 *   type (ties to even), value read back = code * scale.
 * +-inf saturates to +-Q; NaN is kept by e4m3 and stored as 0 by int8.
 *   k, v              codes, [B, Hkv, Lmax, d], one byte each;
 *   k_scale, v_scale  fp32 [B, Hkv, ceil(Lmax / block)];
 *   k_tail, v_tail    bf16 [B, Hkv, 2, block, d]: the rows of a sequence's last
 *                     two blocks as they were given (slot = block index mod 2).
 * The tails make the cache a function of the tokens it holds: appending in
 * pieces gives bit for bit what appending at once gives, and the latest append
 * may be taken back in part or whole (rejected drafts).
 * Nothing has to be initialised: what lies past a sequence's length is never
 * used, whatever it holds.
 * Supported: d in {64, 128}, block in {64, 128}, 1 <= Lmax <= 2^30,
 * B * Hkv <= 2^20.  k, v 16-byte, scales 4-byte, tails 32-byte aligned (so the
 * slices of one sequence of a batch are a cache too).
 */
typedef struct {
    int B, Hkv, Lmax, d;
    int block;
    int type; /* logo_cache_type */
    void *k, *v;
    float *k_scale, *v_scale;
    logo_bf16 *k_tail, *v_tail;
} logo_cache8;

/*
 * Writes new tokens into the cache, quantised.  The new rows lie in k and v as
 * the forward pass's do: shape->L new tokens for each of shape->B == cache->B
 * sequences ([B, Hkv, L, d]), or packed ([1, Hkv, T, d], shape->nseq == cache->B
 * sequences; a length may be 0).  shape->Hkv and shape->d equal the cache's;
 * shape->Hq is not used beyond its own check.
 *   start    int32 [B] (device): sequence b's rows go to positions start[b] ..
 *            start[b] + n_b - 1, so that start[b] + n_b becomes its length.
 *            start[b] may be the length so far, any multiple of `block` up to it,
 *            or, where the sequence's latest append went from s to e, a position
 *            from s to e whose block is one of the last two up to e.  Positions
 *            behind the new rows are given up, also where n_b is 0 (every draft
 *            rejected): the cache is then the one of the first start[b] tokens.
 *   new_len  int32 [B] (device) receiving start[b] + n_b, or NULL; apart from start.
 * k and v must be 32-byte aligned.  A sequence whose rows do not fit (start < 0
 * or start + n_b > Lmax), or whose packed offsets are out of order, beyond T or
 * longer than max_seqlen, is left as it is (new_len = start) and reported:
 * logo_check gives LOGO_ERR_INVALID_ARG.  The workspace (256 bytes are enough)
 * carries the status word only.  2 * B * Hkv times the blocks that the longest
 * sequence can touch must stay below 2^31 (LOGO_ERR_UNSUPPORTED).
 */
LOGO_API logo_status logo_cache8_append(const logo_cache8 *cache, const logo_bf16 *k, const logo_bf16 *v,
                                        const logo_shape *shape, const int32_t *start, int32_t *new_len, void *ws,
                                        size_t ws_bytes, logo_stream_t stream);

/*
 * Reads rows back: k_out and v_out receive the values (code * scale, rounded
 * once to bf16) of positions start[b] .. start[b] + n_b - 1 of every sequence,
 * laid out as `shape` says ([B, Hkv, L, d], or packed [1, Hkv, T, d]; rows of a
 * packed tensor that lie in no sequence are left as they were).  The positions
 * must have been written; the call does not know the lengths.  Outputs must be
 * 32-byte aligned.  Errors as for logo_cache8_append.
 */
LOGO_API logo_status logo_cache8_read(const logo_cache8 *cache, const int32_t *start, const logo_shape *shape,
                                      logo_bf16 *k_out, logo_bf16 *v_out, void *ws, size_t ws_bytes,
                                      logo_stream_t stream);

/*
 * Decode step over the cache: what logo_decode computes, with keys and values
 * the cache's (code * scale), for n >= 1 new tokens a sequence.  Token i of
 * sequence b sits at position t = cache_len[b] - n + i (all n are already
 * written there):
 *   local  = softmax attention over positions max(0, t - W + 1) .. t;
 *   global = softmax attention over 0 .. t, only when gate[b, i] > *tau
 *            (never for NaN);
 *   out    = local + sigmoid(gate[b, i]) * global, or local; zero where t < 0.
 * Positions before every window are read only for sequences with a token that
 * takes the global branch.
 *   q, out     [B, Hq, n, d] bf16;  gate fp32 [B, n];  tau one fp32;
 *   cache_len  int32 [B] (device, 0 <= cache_len <= Lmax; another value reads
 *              nothing, gives a zero output and is reported by logo_check as
 *              LOGO_ERR_INVALID_ARG);
 *   selected   int32 [B, n] (device; 1 iff gate > *tau) or NULL.
 * Hq / Hkv * n must not exceed 32.  The workspace must hold
 * logo_decode8_workspace_size(cache, Hq, n) bytes (0 if they are not supported),
 * be set up once with logo_workspace_init, and be used by one stream (or one
 * captured graph) at a time.
 * A key, value or scale that is not finite reaches the tokens that attend to its
 * position (a scale's: its block) and no others; a value's scale that is not
 * finite makes their outputs NaN.
 */
LOGO_API size_t logo_decode8_workspace_size(const logo_cache8 *cache, int Hq, int n);
LOGO_API logo_status logo_decode8(const logo_bf16 *q, const logo_cache8 *cache, const int32_t *cache_len,
                                  const float *gate, const float *tau, int Hq, int n, int window, float scale,
                                  logo_bf16 *out, int32_t *selected, void *ws, size_t ws_bytes, logo_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LOGO_CACHE8_H_ */
