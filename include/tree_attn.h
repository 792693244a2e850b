/*
 * tree_attn.h -- C ABI of the attention that verifies a tree of drafted tokens
 * over a paged key/value cache.
 *
 * Each of B requests has a context of lens[b] tokens in the cache and T drafted
 * tokens after it, whose keys and values the caller has written at positions
 * lens[b] .. lens[b] + T - 1.  The drafts form a tree: bit j of tree_mask[b][i]
 * says that draft i attends to draft j (itself and its ancestors; T = 1 with
 * mask 1 is plain decoding).  Query head h reads kv head h * Hkv / Hq:
 *
 *   see(b, i, p) = p < lens[b], or p = lens[b] + j and bit j of tree_mask[b][i]
 *   a_p          = scale * q[b][i][h] . k[p]      over the p that it sees
 *   out[b][i][h] = sum_p exp(a_p) v[p] / sum_p exp(a_p)
 *   lse[b][i][h] = log sum_p exp(a_p)
 *
 * A row that sees nothing gets out = 0 and lse = -infinity.  What a row does not
 * see has no influence on it, NaN and infinity included.
 *
 * Statuses, dtypes, streams, ownership, capture and workspaces are those of
 * w4a16.h: device pointers 16-byte aligned (block_table, lens and tree_mask
 * need their own type's alignment only), arguments checked on the host before
 * anything is enqueued, no allocation, no synchronization.
 */
#ifndef TREE_ATTN_H
#define TREE_ATTN_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* q           [B*T][Hq][D], q_stride elements from token to token (>= Hq * D, a
 *             multiple of 8: the rows of a fused qkv product can be passed as they are)
 * k, v        the cache: element d of head h of token s of page p at
 *             p * page_stride + s * token_stride + h * head_stride + d, the same
 *             for both (64-bit; non-negative multiples of 8).  Any order of tokens and heads.
 * block_table int32 [B][table_stride]: page of positions [i * page_size, (i+1) * page_size).
 *             Entries outside 0 .. num_pages - 1 are taken as the nearest of them.
 * lens        int32 [B], read on the device; taken as 0 .. max_len
 * tree_mask   uint64 [B][T]
 * out         [B*T][Hq][D], contiguous, of dtype; lse fp32 [B*T][Hq] or NULL
 * dtype       W4A16_F16 or W4A16_BF16, of q, k, v and out.  Products and sums
 *             are fp32; the probabilities take the dtype for the product with v.
 * Shape: B >= 1, 1 <= T <= 64, Hq a multiple of Hkv, Hq <= 2^16, B * Hq <= 2^24, D 64, 128
 * or 256, page_size a power of two with page_size * token_stride < 2^30, 0 <= max_len <= 2^30, table_stride * page_size >=
 * max_len + T.  max_len bounds lens (host knowledge: it sizes the split over the
 * keys; a captured graph stays valid for every lens up to it).  Deterministic
 * for the same lens.  workspace may be NULL where the query reports 0.  Both calls
 * return W4A16_ERR_UNSUPPORTED for another D, and where a launch would need 2^32
 * work-items (at the earliest with 2^24 pairs of a request and a kv head, or 2^28 rows B * T * Hq). */
int tree_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int max_len, size_t* bytes);
int tree_attn(const void* q, long long q_stride, const void* k, const void* v, int dtype,
              int num_pages, int page_size, long long page_stride, long long token_stride,
              long long head_stride, const int32_t* block_table, int table_stride,
              const int32_t* lens, int max_len, const uint64_t* tree_mask, float scale, void* out,
              float* lse, int B, int T, int Hq, int Hkv, int D, void* workspace,
              size_t workspace_bytes, w4a16_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TREE_ATTN_H */
