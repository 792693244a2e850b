/*
 * w8a8.h -- C ABI of the 8-bit block-scaled layer: RMS norm and gated product
 * with 8-bit outputs, and the matrix product that takes them.
 *
 * 8 bits are OCP E4M3 ("e4m3fn": 1 sign, 4 exponent, 3 mantissa bits, largest
 * value 448, no infinity, NaN = 0x7f).  Each 128 consecutive k of a row share
 * one fp32 scale (the last group of a row may be shorter); each 128 x 128 block
 * of the weights shares one:
 *   x         e4m3 [M][K], row-major, contiguous
 *   x_scales  fp32 [ceil(K/128)][M]        x[m][k] stands for x * x_scales[k/128][m]
 *   w         e4m3 [N][K], row-major, contiguous (a layer's own layout, not packed)
 *   w_scales  fp32 [ceil(N/128)][ceil(K/128)]
 *
 * Statuses, dtypes, streams, alignment, ownership, capture and workspaces are
 * those of w4a16.h: device pointers 16-byte aligned, arguments checked on the
 * host before anything is enqueued, no allocation, no synchronization, one
 * workspace (its head zeroed once) for all calls on one stream.
 */
#ifndef W8A8_H
#define W8A8_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* h = x + residual (fp32; h = x where residual is NULL)
 * n = h / sqrt(mean_k(h^2) + eps) * weight, from the fp32 h
 * For each row and each 128 columns: s = max(amax |n|, 2^-60) / 448,
 * q = n / s rounded to nearest even, scales[k/128][m] = s.
 *
 * x [M][K] with ldx elements from row to row (ldx >= K, a multiple of 8);
 * residual and h_out [M][K] contiguous, both residual_dtype; weight [K]; y_out
 * [M][K] contiguous gets n in y_dtype (for a layer with 16-bit x, such as
 * w4a16_gemv's).  dtypes: x f16 or bf16 or f32, and so are the others.
 * residual may be NULL (h_out then has to be NULL too), h_out may be NULL or
 * the residual itself (updated in place); y_out or the pair q, scales may be NULL,
 * not both.  Otherwise nothing overlaps.  Shape: M >= 1, 16 <= K <= 32768,
 * K % 16 == 0; eps finite and >= 0.  A longer K returns W4A16_ERR_UNSUPPORTED, and
 * so does a launch of 2^32 work-items (a row takes one for each 8 columns up to 1024,
 * 64 at least: M from 2^26 where K <= 512, at the earliest from 2^22).
 * A row with a NaN gives NaN throughout, one with an infinity NaN in its
 * block, as the formula does in fp32. */
int w8a8_rmsnorm_quant(const void* x, int x_dtype, long long ldx, const void* residual,
                       int residual_dtype, void* h_out, const void* weight, int weight_dtype,
                       float eps, void* y_out, int y_dtype, void* q, float* scales, int M, int K,
                       w4a16_stream_t stream);

/* n[m][k] = silu(x[m][k]) * x[m][K + k], silu(g) = g / (1 + exp(-g)), in fp32;
 * then q, scales and y_out as above.  x [M][2K] (the fused gate/up product)
 * with ldx elements from row to row (ldx >= 2K, a multiple of 8), x_dtype f16, bf16 or
 * f32.  Shape: M >= 1, 16 <= K <= 2^30, K % 16 == 0, M * ceil(K/2048) < 2^31; a
 * launch of 2^32 work-items (a row takes one for each 8 columns, a power of two of them and
 * 16 at least up to K = 2048, then whole 256s) returns W4A16_ERR_UNSUPPORTED. */
int w8a8_silu_mul_quant(const void* x, int x_dtype, long long ldx, void* y_out, int y_dtype,
                        void* q, float* scales, int M, int K, w4a16_stream_t stream);

/* y[m][n] = sum_b x_scales[b][m] w_scales[n/128][b] sum_{k in block b} x[m][k] w[n][k]
 *
 * Products run on the e4m3 matrix unit, which adds eight consecutive k aligned
 * to their largest product (what lies below 2^-13 of it is dropped: about 2e-6 of
 * the sum of magnitudes, far under what 8-bit operands carry) and keeps the
 * sums of those in fp32.  Sums over blocks are fp32, the scales' product is
 * formed in fp32 once per row and block; the result is deterministic.
 * y [M][N] contiguous, y_dtype f32, f16 or bf16 (rounded once).  Shape:
 * 1 <= M <= 2^26, N >= 8, N % 8 == 0, 16 <= K <= 2^20, K % 16 == 0.  M is not limited to a
 * few rows: one token to whole prompts.  x, w, y and the workspace do not overlap.
 * workspace may be NULL where w8a8_workspace_bytes reports 0.  Both calls return
 * W4A16_ERR_UNSUPPORTED where a product needs more work-items than a launch takes
 * (2^32 - 1; M * N from about 2^39). */
int w8a8_workspace_bytes(int M, int N, int K, size_t* bytes);
int w8a8_gemm(const void* x, const float* x_scales, const void* w, const float* w_scales, void* y,
              int y_dtype, int M, int N, int K, void* workspace, size_t workspace_bytes,
              w4a16_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H */
