/*
 * rope_append.h -- C ABI of rotary positions and of the append to a paged
 * key/value cache (the one tree_attn.h and prefix_attn.h read).
 *
 * Token m at position p = positions[m] has the query heads q[m][h], the key heads
 * k[m][h] and the value heads v[m][h].  The first rot_dim elements of each query
 * and key head are rotated in rot_dim / 2 pairs, the others stay:
 *
 *   angle_i  = p * inv_freq[i]                     i = 0 .. rot_dim / 2 - 1
 *   (x, y)  -> (x c - y s, y c + x s),             c = gain cos(angle_i), s = gain sin(angle_i)
 *
 * where pair i is elements i and i + rot_dim / 2 (halves) or 2 i and 2 i + 1
 * (interleaved).  The product p * inv_freq[i] is formed and reduced in 64 bits, so
 * far positions keep their angle; sines, cosines and the rotation are fp32, rounded
 * once to the dtype.  Rotated queries go to q_out, rotated keys and the values to
 * slot slots[m] of the cache.
 *
 * Statuses, dtypes, streams, ownership and capture are those of w4a16.h: device
 * pointers 16-byte aligned (positions, inv_freq and slots need their own type's
 * alignment only), arguments checked on the host before anything is enqueued, no
 * allocation, no synchronization.
 */
#ifndef ROPE_APPEND_H
#define ROPE_APPEND_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Host only: inv_freq[i] = base^(-2 i / rot_dim), i < rot_dim / 2, in HOST memory,
 * scaled for contexts `factor` times as long as the ones a model was trained on:
 *   original = 0: all divided by factor (positions interpolated; factor 1: as they are)
 *   original > 0 (that length): by parts.  A pair that turns n = original f / (2 pi) times
 *     over the length keeps f where n >= fast, gets f / factor where n <= slow, and
 *     f (w + (1 - w) / factor), w = (n - slow) / (fast - slow), between.
 * The ramp is linear in the turns.  A model with another one (linear in the pair's index, say: single
 * frequencies differ by up to two fifths) needs its own list, made by its own formula: rope_append takes any.
 * rot_dim even, 2..1024; base > 1, factor >= 1, original >= 0, and 0 < slow < fast
 * where original > 0; all finite. */
int rope_frequencies(float* inv_freq, int rot_dim, double base, double factor, double original,
                     double slow, double fast);

/* q         [M][Hq][D], q_stride elements from token to token (>= Hq * D); k, v [M][Hkv][D]
 *           likewise.  Strides are multiples of 8, so the parts of a fused qkv product's
 *           rows can be passed as they are.
 * positions int32 [M], any sign; inv_freq fp32 [rot_dim / 2].  Both NULL where rot_dim = 0.
 * q_out     [M][Hq][D] with q_out_stride; may be q itself (same stride: rotated in place)
 * k_cache, v_cache  element d of head h of token s of page p at p * page_stride +
 *           s * token_stride + h * head_stride + d, the same for both (64-bit; non-negative
 *           multiples of 8), as in tree_attn.h
 * slots     int64 [M]: page * page_size + token.  A slot outside 0 .. num_pages * page_size - 1
 *           (-1 for the rows that fill up a captured batch) appends nothing; its q is
 *           rotated all the same.  Slots of one call are distinct: of two rows with the same slot
 *           either may be stored, or parts of both.
 * interleaved 0 (halves) or 1; gain finite, multiplies c and s; dtype W4A16_F16 or W4A16_BF16.
 * q and q_out may both be NULL (only keys and values: Hq is not looked at); k, v, both caches and slots
 * may all be NULL (only queries: Hkv, the page counts and strides are not).  Not both.  Other than q_out = q nothing overlaps.
 * Shape: M >= 1, D a multiple of 16 up to 512, rot_dim a multiple of 16 up to D (a thread turns the eight pairs that two
 * 16-byte pieces of a head hold, so no piece is part turned; 20 or 24 elements are refused), 1 <= Hq, Hkv
 * <= 2^16, page_size a power of two.  A launch of 2^32 work-items (a token takes 64 at
 * least, and about one for each 16 or, of many tokens, 64 elements of its heads) returns
 * W4A16_ERR_UNSUPPORTED. */
int rope_append(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                long long v_stride, int dtype, const int32_t* positions, const float* inv_freq,
                int rot_dim, int interleaved, float gain, void* q_out, long long q_out_stride,
                void* k_cache, void* v_cache, int num_pages, int page_size, long long page_stride,
                long long token_stride, long long head_stride, const int64_t* slots, int M, int Hq,
                int Hkv, int D, w4a16_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_APPEND_H */
