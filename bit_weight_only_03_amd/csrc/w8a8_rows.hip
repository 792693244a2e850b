// w8a8_rows.hip -- the row operators of the 8-bit layer: RMS norm with the
// residual's addition, and the gated product, both with e4m3 output and one
// fp32 scale for each 128 columns of a row.
//
// Both are one pass over memory: every element is loaded once, lives in
// registers as fp32 until its row's (or block's) statistic is known, and is
// stored once.  Eight consecutive elements belong to a lane, so the 16 lanes
// of a DPP row hold exactly one block of 128 columns and its largest
// magnitude takes four DPP steps, no LDS.
#include "w8a8_common.h"

using namespace w4k;

namespace {

struct NormArgs {
    const void* x;
    const void* residual;
    const void* weight;
    void* h;
    void* y;
    uint8_t* q;
    float* scales;
    long long ldx;
    int x_dtype, residual_dtype, weight_dtype, y_dtype;
    int M, K;
    float eps;
};

// The sum over a wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// P vectors of 8 columns per lane: vector p of the row's lane t is number
// p * threads + t, so a wave's loads are contiguous and a block of 128 columns
// stays inside 16 lanes (threads is a multiple of 64).  Where K / 8 vectors do
// not fill the last ones, those lanes load nothing and add zeros.  A row per
// workgroup, its waves' sums joined through LDS (a wave per row and four rows
// per workgroup took as long for K = 256 .. 1024).  NT: results bypass the
// caches' retention where they are larger than what the next kernel could find
// there (2560 x 16384: 55 against 62 us; 8192 x 5120: 65 against 67; 2048 x 5120,
// below the limit, 16.1 against 16.5, but there the next kernel finds them).
// Bound by memory: 8192 x 5120 with residual moves 295 MB in 65 us, 4.5 TB/s,
// where a 1 GiB copy reaches 4.8.  More vectors per lane and fewer waves were
// slower (when P = 1 took 67 us, P = 2 took 70, 4: 84, 10: 103): they only delay the first store.
template <int P, bool NT>
__global__ __launch_bounds__(1024) void rmsnorm_quant_kernel(NormArgs a) {
    const int t = threadIdx.x, threads = blockDim.x;
    const size_t row = blockIdx.x;
    const int nv = a.K / 8;
    float h[P][8], w[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int v = p * threads + t;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[p][e] = w[p][e] = 0.f;
        if (v < nv) {
            load8(a.x, a.x_dtype, row * (size_t)a.ldx + 8 * (size_t)v, h[p]);
            load8(a.weight, a.weight_dtype, 8 * (size_t)v, w[p]);
        }
    }
    if (a.residual) {
        float r[P][8];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int v = p * threads + t;
#pragma unroll
            for (int e = 0; e < 8; ++e) r[p][e] = 0.f;
            if (v < nv) load8(a.residual, a.residual_dtype, row * a.K + 8 * (size_t)v, r[p]);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int v = p * threads + t;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[p][e] += r[p][e];
            if (a.h && v < nv) store8<NT>(a.h, a.residual_dtype, row * a.K + 8 * (size_t)v, h[p]);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[p][e], h[p][e], ss);
    ss = wave_sum(ss);
    __shared__ float part[16];
    if ((t & 63) == 0) part[t >> 6] = ss;
    __syncthreads();
    float total = 0.f;
    for (int i = 0; i < threads >> 6; ++i) total += part[i];
    const float rstd = 1.0f / __builtin_sqrtf(total / (float)a.K + a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int v = p * threads + t;
        float n[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = h[p][e] * rstd * w[p][e];
        if (a.y && v < nv) store8<NT>(a.y, a.y_dtype, row * a.K + 8 * (size_t)v, n);
        if (a.q) {
            // Lanes past the row's end hold zeros: they leave the maximum as it is.
            const float s = block_scale(n);
            if (v < nv) {
                store_q8<NT>(a.q + row * a.K + 8 * (size_t)v, n, s);
                if ((t & 15) == 0) a.scales[(size_t)(v >> 4) * a.M + row] = s;
            }
        }
    }
}

// g / (1 + exp(-g)) from the hardware's 2^t and reciprocal (about one ulp
// each; IEEE division and expf would make the operator bound by the VALU).
// t = -g log2(e) is taken in two pieces, the rounding of the product and the
// rest of the constant, so that 2^t keeps its relative error for large |g|.
// exp(-g) past fp32's range is infinite and the result 0, as in the formula.
// The reciprocal unit flushes a result below 2^-126 to zero, so it takes
// (1 + p) / 16: 1 / (1 + p) is subnormal from g = -87.3 on, its product with g is not
// (4096 x 17408: 68.3 us against 67.4 without; a branch for such waves took as long).
__device__ __forceinline__ float silu(float g) {
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
    const float t = -g * kLog2e;
    const float rest = __builtin_fmaf(-g, kLog2eRest, __builtin_fmaf(-g, kLog2e, -t));
    float p = __builtin_amdgcn_exp2f(t);
    // Not where p is 0 or infinite: there the correction could be 0 * inf.
    const float c = p * (kLn2 * rest);
    p = __builtin_fabsf(t) < 128.0f ? p + c : p;
    return g * (__builtin_amdgcn_rcpf(__builtin_fmaf(p, 0x1p-4f, 0x1p-4f)) * 0x1p-4f);
}

struct GatedArgs {
    const void* x;
    void* y;
    uint8_t* q;
    float* scales;
    long long ldx;
    int x_dtype, y_dtype;
    int M, K;
    int chunks;   // workgroups per row
    int shift;    // log2 of the lanes that take a row
};

constexpr int kGatedThreads = 256;
constexpr int kGatedCols = kGatedThreads * 8;

// A workgroup takes 2048 columns of one row, or several short rows (a power of
// two of lanes each, 16 at least); a block of 128 columns is 16 lanes.  Bound by
// memory: 4096 x 17408 moves 359 MB in 68 us, 5.3 TB/s, with results stored past
// the caches or not.
template <bool NT>
__global__ __launch_bounds__(kGatedThreads) void silu_mul_quant_kernel(GatedArgs a) {
    const unsigned chunk = blockIdx.x % (unsigned)a.chunks;
    const size_t row = (size_t)(blockIdx.x / (unsigned)a.chunks) * (kGatedThreads >> a.shift) + (threadIdx.x >> a.shift);
    if (row >= (size_t)a.M) return;   // whole blocks of lanes
    const int k = chunk * kGatedCols + (int)(threadIdx.x & ((1u << a.shift) - 1)) * 8;
    float g[8], u[8], n[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.f;
    if (k < a.K) {
        load8(a.x, a.x_dtype, row * (size_t)a.ldx + k, g);
        load8(a.x, a.x_dtype, row * (size_t)a.ldx + a.K + k, u);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = silu(g[e]) * u[e];
    if (a.y && k < a.K) store8<NT>(a.y, a.y_dtype, row * a.K + k, n);
    if (a.q) {
        const float s = block_scale(n);
        if (k < a.K) {
            store_q8<NT>(a.q + row * a.K + k, n, s);
            if ((threadIdx.x & 15) == 0) a.scales[(size_t)(k >> 7) * a.M + row] = s;
        }
    }
}

bool dtype_ok(int d) { return d == W4A16_F16 || d == W4A16_BF16 || d == W4A16_F32; }

constexpr size_t kStreamElements = (size_t)16 << 20;   // results from here on are stored past the caches
constexpr int kMaxThreads = 1024;
constexpr int kMaxNormPasses = 4;
constexpr int kMaxNormK = kMaxThreads * 8 * kMaxNormPasses;

// Output checks shared by the row operators: y, or q with its scales, or all.
int check_out(const void* y, int y_dtype, const void* q, const float* scales) {
    if (!y && !q) return W4A16_ERR_NULL;
    if (!q != !scales) return W4A16_ERR_NULL;
    if (y && !dtype_ok(y_dtype)) return W4A16_ERR_DTYPE;
    if (!w4h::aligned16(y) || !w4h::aligned16(q) || !w4h::aligned16(scales)) return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

}  // namespace

extern "C" int w8a8_rmsnorm_quant(const void* x, int x_dtype, long long ldx, const void* residual,
                                  int residual_dtype, void* h_out, const void* weight,
                                  int weight_dtype, float eps, void* y_out, int y_dtype, void* q,
                                  float* scales, int M, int K, w4a16_stream_t stream) {
    if (!x || !weight || (h_out && !residual)) return W4A16_ERR_NULL;
    if (!dtype_ok(x_dtype) || !dtype_ok(weight_dtype) || (residual && !dtype_ok(residual_dtype)))
        return W4A16_ERR_DTYPE;
    if (M < 1 || K < 16 || K % 16 || ldx < K || ldx % 8 || !(eps >= 0.f) || eps > 3.4e38f)
        return W4A16_ERR_SHAPE;
    if (!w4h::aligned16(x) || !w4h::aligned16(residual) || !w4h::aligned16(h_out) ||
        !w4h::aligned16(weight))
        return W4A16_ERR_ALIGN;
    if (int rc = check_out(y_out, y_dtype, q, scales)) return rc;
    if (K > kMaxNormK) return W4A16_ERR_UNSUPPORTED;
    NormArgs a{x, residual, weight, h_out, y_out, (uint8_t*)q, scales, ldx, x_dtype,
               residual_dtype, weight_dtype, y_dtype, M, K, eps};
    const int nv = K / 8;
    const bool nt = (size_t)M * K >= kStreamElements;
    const int P = nv <= kMaxThreads ? 1 : nv <= 2 * kMaxThreads ? 2 : 4;
    const int threads = (((nv + P - 1) / P) + 63) / 64 * 64;
    if ((long long)M * threads > kMaxLanes) return W4A16_ERR_UNSUPPORTED;
    auto kernel = P == 1   ? (nt ? rmsnorm_quant_kernel<1, true> : rmsnorm_quant_kernel<1, false>)
                  : P == 2 ? (nt ? rmsnorm_quant_kernel<2, true> : rmsnorm_quant_kernel<2, false>)
                           : (nt ? rmsnorm_quant_kernel<4, true> : rmsnorm_quant_kernel<4, false>);
    w4h::begin_launches();
    hipLaunchKernelGGL(kernel, dim3(M), dim3(threads), 0, (hipStream_t)stream, a);
    w4h::note_variant("w8a8_%s passes=%lld threads=%lld rows=%lld", "rmsnorm", P, threads, M);
    return w4h::launch_status();
}

extern "C" int w8a8_silu_mul_quant(const void* x, int x_dtype, long long ldx, void* y_out,
                                   int y_dtype, void* q, float* scales, int M, int K,
                                   w4a16_stream_t stream) {
    if (!x) return W4A16_ERR_NULL;
    if (!dtype_ok(x_dtype)) return W4A16_ERR_DTYPE;
    if (M < 1 || K < 16 || K % 16 || K > (1 << 30) || ldx < 2LL * K || ldx % 8) return W4A16_ERR_SHAPE;
    if (!w4h::aligned16(x)) return W4A16_ERR_ALIGN;
    if (int rc = check_out(y_out, y_dtype, q, scales)) return rc;
    const long long chunks = (K + kGatedCols - 1) / kGatedCols;
    if (chunks * M > 0x7fffffffLL) return W4A16_ERR_SHAPE;
    int shift = 4;   // 16 lanes: 128 columns
    while (shift < 8 && (8 << shift) < K) ++shift;
    const long long groups = (M + (kGatedThreads >> shift) - 1LL) / (kGatedThreads >> shift);
    GatedArgs a{x, y_out, (uint8_t*)q, scales, ldx, x_dtype, y_dtype, M, K, (int)chunks, shift};
    const bool nt = (size_t)M * K >= kStreamElements;
    if (chunks * groups * kGatedThreads > kMaxLanes) return W4A16_ERR_UNSUPPORTED;
    w4h::begin_launches();
    hipLaunchKernelGGL((nt ? silu_mul_quant_kernel<true> : silu_mul_quant_kernel<false>), dim3((unsigned)(chunks * groups)),
                       dim3(kGatedThreads), 0, (hipStream_t)stream, a);
    w4h::note_variant("w8a8_%s chunks=%lld rows=%lld", "silu_mul", chunks, M);
    return w4h::launch_status();
}
