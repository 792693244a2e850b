/*
 * lora.h -- C ABI of low-rank adapters of many requests beside a shared
 * projection (the result of any of the library's products).
 *
 * n_adapters adapters are held next to the projection's weights.  Row m uses
 * adapter a = adapter[m], with rank r = ranks[a] and scale s = scales[a].  The N
 * columns of a fused projection (q, k, v or gate, up) are `parts` ranges of columns,
 * each with an A of its own; p(n) is the part of column n:
 *
 *   h[m][p][j] = sum_k a[a][p][j][k] x[m][k]                                  j < r
 *   y[m][n]    = base[m][n] + s sum_{j < r} b[a][n][j] h[m][p(n)][j]
 *
 * A row whose adapter is outside 0 .. n_adapters - 1 (-1: none) gets y = base.
 * Rows of one adapter may lie anywhere in the batch; in large batches they cost less side by side (an adapter is
 * read again by every tile of 16 or 64 rows that uses it).
 *
 * Statuses, dtypes, streams, ownership, capture and workspaces are those of
 * w4a16.h: device pointers 16-byte aligned (ranks, scales and adapter need their own
 * type's alignment only), arguments checked on the host before anything is
 * enqueued, no allocation, no synchronization.
 */
#ifndef LORA_H
#define LORA_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_MAX_PARTS 4

/* x          [M][K] with ldx elements from row to row (ldx >= K, a multiple of 8)
 * a          [n_adapters][parts][R][K], contiguous
 * b          [n_adapters][N][R], contiguous
 * ranks      int32 [n_adapters], read on the device and taken as 0 .. R; NULL: all R.  Up to the next
 *            multiple of 8 a and b hold zeros; what lies behind it is not read.
 * scales     fp32 [n_adapters], or NULL: all 1
 * adapter    int32 [M]
 * base, y    [M][N] of y_dtype (f32, f16 or bf16), ldy elements from row to row
 *            (ldy >= N, a multiple of 8).  base may be y (updated in place) or NULL (zeros).
 * part_cols  HOST array of `parts` widths that add up to N; all but the last are
 *            multiples of 64.  NULL where parts is 1.
 * dtype      W4A16_F16 or W4A16_BF16, of x, a and b.  Products and sums are fp32; h stays fp32
 *            (it enters the second product as a sum of 16-bit terms: 2^-16 of its
 *            largest element at most is left out for a 16-bit y, 2^-21 for an fp32 y).
 * The result is deterministic.  A row with a NaN or an infinity changes no other row.  An infinity in x or a makes an
 * infinite sum infinite; b is finite (an infinity there makes its column NaN for its adapter's rows, as h's terms may be 0).
 * Other than base = y nothing overlaps.
 * Shape: 1 <= M <= 2^26, N >= 8, N % 8 == 0, N <= 2^24, 8 <= K <= 2^20, K % 8 == 0, ldx <= 2^24, ldy <= 2^25,
 * R a multiple of 8 up to 256, 1 <= n_adapters, 1 <= parts <= 4.  workspace may be NULL where the query
 * reports 0; what it reports for M rows (the other sizes the same) is enough for any fewer.  Both calls return W4A16_ERR_UNSUPPORTED where a launch would need 2^32 work-items. */
int lora_workspace_bytes(int M, int N, int K, int R, int parts, size_t* bytes);
int lora_add(const void* x, int dtype, long long ldx, const void* a, const void* b,
             const int32_t* ranks, const float* scales, int n_adapters, const int32_t* adapter,
             const void* base, void* y, int y_dtype, long long ldy, const int* part_cols, int parts,
             int M, int N, int K, int R, void* workspace, size_t workspace_bytes,
             w4a16_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_H */
