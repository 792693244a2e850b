// rope_append.hip -- rotary positions, and keys and values appended to a paged
// cache, in one pass over the rows of a fused qkv product: pair (x, y) of a query or key
// head at position p becomes (x c - y s, y c + x s), c and s the cosine and sine of p f.
//
// Bound by memory: 64 operations for 32 bytes read and written.  8192 tokens of 40 query and
// 8 key/value heads of 128 (235 MB) take 48.8 us, 4.8 TB/s; a plain copy reaches 5.2.  One
// token takes 2.8 us in a graph, a launch's time.  So nothing is read twice, accesses are 16
// bytes wide and all of a thread's are on their way before the first is used; the sines, 64-bit work, are
// made once per token and not once per head.
#include <math.h>

#include "w8a8_common.h"
#include "../../include/rope_append.h"

using namespace w4k;

namespace {

constexpr int kMaxD = 512;
constexpr int kMaxThreads = 1024;
// With a thread for each 16 elements: from here on a thread takes four heads, whose loads it has in flight
// together (40/8 heads of 128, 1024 tokens: 6.8 us with four, 6.2 with one; 2048: 9.4, 10.3; 4096: 20.0, 20.7).
constexpr long long kManyThreads = 3 << 18;

struct RopeArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int* positions;
    const float* freq;
    uint16_t* q_out;
    uint16_t* k_cache;
    uint16_t* v_cache;
    const long long* slots;
    long long q_stride, k_stride, v_stride, q_out_stride;
    long long page_stride, token_stride, head_stride, num_slots;
    int page_shift;
    int half;            // pairs that are rotated
    float gain;
    int Hq, Hkv, H;      // H: query, key and value heads of a token
    int items;           // threads of a head, 16 elements each
    int heads;           // heads that a workgroup takes at once
    int chunks;          // workgroups of a token
};

// cos and sin of p f.  The angle in quarter turns is a 64-bit product (p and f
// have 31 and 24 bits: what it loses is 2^-53 of it, below 2^-33 turns up to
// position 2^20), its fraction is exact.  |x| <= pi / 4 then: the Taylor sums up to
// x^9 and x^10 leave out less than 2^-29.
__device__ __forceinline__ float2 turn(int p, float f, float gain) {
    constexpr double kQuarters = 0x1.45f306dc9c883p-1;   // 2 / pi
    const double a = (double)p * (double)f * kQuarters;
    const double n = __builtin_rint(a);
    const float x = (float)(a - n) * 0x1.921fb6p+0f;     // pi / 2
    const int quarter = (int)(n - 4.0 * __builtin_rint(n * 0.25)) & 3;
    const float z = x * x;
    float s = __builtin_fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
    s = __builtin_fmaf(z, s, 1.0f / 120.0f);
    s = __builtin_fmaf(z, s, -1.0f / 6.0f);
    s = __builtin_fmaf(x * z, s, x);
    float c = __builtin_fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    c = __builtin_fmaf(z, c, -1.0f / 720.0f);
    c = __builtin_fmaf(z, c, 1.0f / 24.0f);
    c = __builtin_fmaf(z, c, -0.5f);
    c = __builtin_fmaf(z, c, 1.0f);
    const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
    return float2{(quarter == 1 || quarter == 2 ? -cc : cc) * gain, (quarter & 2 ? -ss : ss) * gain};
}

template <bool BF16>
__device__ __forceinline__ float low(uint32_t v) {
    return BF16 ? bitcast<float>(v << 16) : f16_bits_to_f32((uint16_t)v);
}
template <bool BF16>
__device__ __forceinline__ float high(uint32_t v) {
    return BF16 ? bitcast<float>(v & 0xffff0000u) : f16_bits_to_f32((uint16_t)(v >> 16));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack(float a, float b) {
    return BF16 ? pk_bf16(a, b) : pk_f16(a, b);
}

// A workgroup takes one token: its first threads make the cosines and sines of
// the pairs, once for all heads, while every thread's elements are on their way.
// A thread takes 16 elements of a head, as two 16-byte chunks that hold eight
// whole pairs: chunks i and i + rot/16 (halves) or 2 i and 2 i + 1 (interleaved).
// P heads per thread, all loaded before the first is needed.  A token with more heads than
// 1024 threads take has several workgroups.
template <bool BF16, bool HALVES, int P>
__global__ __launch_bounds__(kMaxThreads) void rope_append_kernel(RopeArgs a) {
    __shared__ __attribute__((aligned(16))) float cs[kMaxD / 2], sn[kMaxD / 2];
    const uint32_t chunk = blockIdx.x % (uint32_t)a.chunks;
    const size_t m = blockIdx.x / (uint32_t)a.chunks;
    const int t = threadIdx.x, item = t % a.items, in_pass = t / a.items, head0 = chunk * a.heads * P + in_pass;
    const int turned = a.half / 8;                                     // items that hold pairs
    const bool rot = item < turned;
    const int c0 = HALVES && rot ? item : 2 * item, c1 = HALVES && rot ? item + turned : 2 * item + 1;
    const long long slot = a.slots ? a.slots[m] : -1;
    const bool append = slot >= 0 && slot < a.num_slots;
    const bool mine = in_pass < a.heads;   // the last wave's other threads help with the sines alone
    u32x4_t x[P], y[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int h = head0 + i * a.heads;
        if (mine && h < a.H && (h < a.Hq || append)) {
            const int kh = h - a.Hq, vh = kh - a.Hkv, d = a.items * 16;
            const uint16_t* const src = kh < 0   ? a.q + m * a.q_stride + (size_t)h * d
                                        : vh < 0 ? a.k + m * a.k_stride + (size_t)kh * d
                                                 : a.v + m * a.v_stride + (size_t)vh * d;
            x[i] = *(const u32x4_t*)(src + 8 * c0);
            y[i] = *(const u32x4_t*)(src + 8 * c1);
        }
    }
    if (a.half) {
        const int p = a.positions[m];
        for (int i = t; i < a.half; i += blockDim.x) {
            const float2 r = turn(p, a.freq[i], a.gain);
            cs[i] = r.x, sn[i] = r.y;
        }
    }
    __syncthreads();
    float c[8], s[8];
    if (rot) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const float4_t cv = *(const float4_t*)(cs + 8 * item + e), sv = *(const float4_t*)(sn + 8 * item + e);
#pragma unroll
            for (int j = 0; j < 4; ++j) c[e + j] = cv[j], s[e + j] = sv[j];
        }
    }
    const long long page = slot >> a.page_shift, in_page = slot & ((1LL << a.page_shift) - 1);
    const long long at = page * a.page_stride + in_page * a.token_stride;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int h = head0 + i * a.heads;
        if (!mine || h >= a.H || (h >= a.Hq && !append)) continue;
        const int kh = h - a.Hq, vh = kh - a.Hkv;
        if (rot && vh < 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (HALVES) {
                    const float u0 = low<BF16>(x[i][j]), u1 = high<BF16>(x[i][j]), v0 = low<BF16>(y[i][j]), v1 = high<BF16>(y[i][j]);
                    const float c0f = c[2 * j], s0f = s[2 * j], c1f = c[2 * j + 1], s1f = s[2 * j + 1];
                    x[i][j] = pack<BF16>(__builtin_fmaf(u0, c0f, -(v0 * s0f)), __builtin_fmaf(u1, c1f, -(v1 * s1f)));
                    y[i][j] = pack<BF16>(__builtin_fmaf(v0, c0f, u0 * s0f), __builtin_fmaf(v1, c1f, u1 * s1f));
                } else {
                    float u = low<BF16>(x[i][j]), v = high<BF16>(x[i][j]);
                    x[i][j] = pack<BF16>(__builtin_fmaf(u, c[j], -(v * s[j])), __builtin_fmaf(v, c[j], u * s[j]));
                    u = low<BF16>(y[i][j]), v = high<BF16>(y[i][j]);
                    y[i][j] = pack<BF16>(__builtin_fmaf(u, c[4 + j], -(v * s[4 + j])), __builtin_fmaf(v, c[4 + j], u * s[4 + j]));
                }
            }
        }
        uint16_t* const dst = kh < 0   ? a.q_out + m * a.q_out_stride + (size_t)h * a.items * 16
                              : vh < 0 ? a.k_cache + at + kh * a.head_stride
                                       : a.v_cache + at + vh * a.head_stride;
        *(u32x4_t*)(dst + 8 * c0) = x[i];
        *(u32x4_t*)(dst + 8 * c1) = y[i];
    }
}

bool stride_ok(long long stride, int heads, int D) { return stride >= (long long)heads * D && stride % 8 == 0; }

}  // namespace

extern "C" int rope_frequencies(float* inv_freq, int rot_dim, double base, double factor, double original,
                                double slow, double fast) {
    if (!inv_freq) return W4A16_ERR_NULL;
    if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 || !(base > 1.0) || !(factor >= 1.0) || !(original >= 0.0) ||
        isinf(base) || isinf(factor) || isinf(original))
        return W4A16_ERR_SHAPE;
    if (original > 0.0 && !(slow > 0.0 && fast > slow && !isinf(fast))) return W4A16_ERR_SHAPE;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot_dim), turns = original * f / (2.0 * M_PI);
        double w = original > 0.0 ? (turns - slow) / (fast - slow) : 0.0;
        w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
        inv_freq[i] = (float)(f * (w + (1.0 - w) / factor));
    }
    return W4A16_OK;
}

extern "C" int rope_append(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                           long long v_stride, int dtype, const int32_t* positions, const float* inv_freq,
                           int rot_dim, int interleaved, float gain, void* q_out, long long q_out_stride,
                           void* k_cache, void* v_cache, int num_pages, int page_size, long long page_stride,
                           long long token_stride, long long head_stride, const int64_t* slots, int M, int Hq,
                           int Hkv, int D, w4a16_stream_t stream) {
    const bool has_q = q || q_out, has_kv = k || v || k_cache || v_cache || slots;
    if (!has_q && !has_kv) return W4A16_ERR_NULL;
    if (has_q && (!q || !q_out)) return W4A16_ERR_NULL;
    if (has_kv && (!k || !v || !k_cache || !v_cache || !slots)) return W4A16_ERR_NULL;
    if (rot_dim && (!positions || !inv_freq)) return W4A16_ERR_NULL;
    if (dtype != W4A16_F16 && dtype != W4A16_BF16) return W4A16_ERR_DTYPE;
    if (M < 1 || D < 16 || D > kMaxD || D % 16 || rot_dim < 0 || rot_dim > D || rot_dim % 16 ||
        (interleaved != 0 && interleaved != 1) || !(gain == gain) || gain - gain != 0.f)
        return W4A16_ERR_SHAPE;
    if (has_q && (Hq < 1 || Hq > (1 << 16) || !stride_ok(q_stride, Hq, D) || !stride_ok(q_out_stride, Hq, D) ||
                  (q == q_out && q_stride != q_out_stride)))
        return W4A16_ERR_SHAPE;
    if (has_kv && (Hkv < 1 || Hkv > (1 << 16) || !stride_ok(k_stride, Hkv, D) || !stride_ok(v_stride, Hkv, D) || num_pages < 1 ||
                   page_size < 1 || (page_size & (page_size - 1)) || page_stride < 0 || token_stride < 0 || head_stride < 0 ||
                   page_stride % 8 || token_stride % 8 || head_stride % 8))
        return W4A16_ERR_SHAPE;
    for (const void* p : {q, k, v, (const void*)q_out, (const void*)k_cache, (const void*)v_cache})
        if (!w4h::aligned16(p)) return W4A16_ERR_ALIGN;
    if (((uintptr_t)positions & 3) || ((uintptr_t)inv_freq & 3) || ((uintptr_t)slots & 7)) return W4A16_ERR_ALIGN;
    RopeArgs a{};
    a.q = (const uint16_t*)q, a.k = (const uint16_t*)k, a.v = (const uint16_t*)v;
    a.positions = positions, a.freq = inv_freq, a.q_out = (uint16_t*)q_out;
    a.k_cache = (uint16_t*)k_cache, a.v_cache = (uint16_t*)v_cache, a.slots = (const long long*)slots;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.q_out_stride = q_out_stride;
    a.page_stride = page_stride, a.token_stride = token_stride, a.head_stride = head_stride;
    a.num_slots = has_kv ? (long long)num_pages * page_size : 0;
    while (has_kv && (1 << a.page_shift) < page_size) ++a.page_shift;
    a.half = rot_dim / 2, a.gain = gain;
    a.Hq = has_q ? Hq : 0, a.Hkv = has_kv ? Hkv : 0, a.H = a.Hq + 2 * a.Hkv;
    a.items = D / 16;
    const bool bf16 = dtype == W4A16_BF16, many = (long long)M * a.H * a.items >= kManyThreads && a.H >= 8;
    const int P = many ? 4 : 1, most = kMaxThreads / a.items, want = (a.H + P - 1) / P;
    a.heads = want < most ? want : most;
    a.chunks = (a.H + a.heads * P - 1) / (a.heads * P);
    const int threads = (a.heads * a.items + 63) / 64 * 64;
    const long long blocks = (long long)M * a.chunks;
    if (blocks * threads > kMaxLanes) return W4A16_ERR_UNSUPPORTED;
    typedef void (*kernel_t)(RopeArgs);
    static const kernel_t kernels[2][2][2] = {
        {{rope_append_kernel<false, true, 1>, rope_append_kernel<false, true, 4>}, {rope_append_kernel<false, false, 1>, rope_append_kernel<false, false, 4>}},
        {{rope_append_kernel<true, true, 1>, rope_append_kernel<true, true, 4>}, {rope_append_kernel<true, false, 1>, rope_append_kernel<true, false, 4>}}};
    w4h::begin_launches();
    hipLaunchKernelGGL(kernels[bf16][interleaved][many], dim3((unsigned)blocks), dim3(threads), 0, (hipStream_t)stream, a);
    w4h::note_variant("%s heads_per_thread=%lld threads=%lld blocks=%lld", "rope_append", P, threads, blocks);
    return w4h::launch_status();
}
