/*
 * prefix_attn.h -- C ABI of attention for a batch whose requests share a long
 * prefix (a system prompt, a document, a block of examples), over a paged
 * key/value cache.
 *
 * The keys and values of the prefix's P = prefix_len[0] tokens lie once in the cache,
 * on the pages of prefix_table.  Each of B requests has a context of its own of
 * lens[b] tokens behind the prefix and T drafted tokens after it, at positions 0 ..
 * lens[b] + T - 1 of its own pages (T = 1 with mask 1 is plain decoding; the tree of
 * drafts is tree_attn.h's).  Query head h reads kv head h * Hkv / Hq:
 *
 *   a_p          = scale * q[b][i][h] . k[p]      over the whole prefix, the request's own context,
 *                                                 and draft j where bit j of tree_mask[b][i] is set
 *   out[b][i][h] = sum_p exp(a_p) v[p] / sum_p exp(a_p)
 *   lse[b][i][h] = log sum_p exp(a_p)
 *
 * The prefix is multiplied once for the rows of all requests together.  A row that
 * sees nothing (no prefix, no context, an empty mask) gets out = 0 and lse = -infinity.  What a
 * row does not see has no influence on it, NaN and infinity included.  An infinity in the values
 * that it sees makes its column infinite however small its probability (both infinities, or a NaN: NaN).
 *
 * Statuses, dtypes, streams, ownership, capture and workspaces are those of
 * w4a16.h: device pointers 16-byte aligned (the tables, lengths and tree_mask need
 * their own type's alignment only), arguments checked on the host before anything is
 * enqueued, no allocation, no synchronization.
 */
#ifndef PREFIX_ATTN_H
#define PREFIX_ATTN_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* q            [B*T][Hq][D], q_stride elements from token to token (>= Hq * D, a
 *              multiple of 8)
 * k, v         the cache, as in tree_attn.h: element d of head h of token s of page p at
 *              p * page_stride + s * token_stride + h * head_stride + d (64-bit; non-negative multiples of 8)
 * prefix_table int32 [ceil(max_prefix / page_size)]: pages of the prefix; may be NULL where max_prefix is 0
 * prefix_len   int32 [1], read on the device; taken as 0 .. max_prefix.  It need not fill its last page.
 * block_table  int32 [B][table_stride]: pages of each request's own positions.
 *              Entries of either table outside 0 .. num_pages - 1 are taken as the nearest of them.
 * lens         int32 [B], read on the device; taken as 0 .. max_len
 * tree_mask    uint64 [B][T]
 * out          [B*T][Hq][D], contiguous, of dtype; lse fp32 [B*T][Hq] or NULL
 * dtype        W4A16_F16 or W4A16_BF16, of q, k, v and out.  Products and sums
 *              are fp32; the probabilities take the dtype for the product with v.
 * Shape: B >= 1, 1 <= T <= 64, Hq a multiple of Hkv, Hq <= 2^16, B * Hq <= 2^24, D 64, 128
 * or 256, page_size a power of two from 16 on with page_size * token_stride < 2^30, 0 <=
 * max_prefix, max_len <= 2^30, table_stride * page_size >= max_len + T.  The maxima bound the
 * lengths (host knowledge: they size the split over the keys; a captured graph stays valid
 * for all lengths up to them).  Deterministic for the same lengths.  workspace may be NULL where the query
 * reports 0; what it reports (at most 128 MiB and the head) is enough for any smaller B, T, max_prefix and max_len
 * too.  A batch whose partial sums pass 128 MiB is taken in several runs of requests that reuse it.
 * Both calls return W4A16_ERR_UNSUPPORTED for another D, the call for a smaller page_size, and both where a launch
 * would need 2^32 work-items. */
int prefix_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int max_prefix, int max_len,
                                size_t* bytes);
int prefix_attn(const void* q, long long q_stride, const void* k, const void* v, int dtype,
                int num_pages, int page_size, long long page_stride, long long token_stride,
                long long head_stride, const int32_t* prefix_table, const int32_t* prefix_len,
                int max_prefix, const int32_t* block_table, int table_stride, const int32_t* lens,
                int max_len, const uint64_t* tree_mask, float scale, void* out, float* lse, int B,
                int T, int Hq, int Hkv, int D, void* workspace, size_t workspace_bytes,
                w4a16_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PREFIX_ATTN_H */
