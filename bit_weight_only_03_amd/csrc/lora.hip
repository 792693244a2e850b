// lora.hip -- low-rank adapters of many requests beside a shared projection:
// y = base + s B (A x), each row with an adapter of its own.
//
// Rows come in tiles of 16, and the distinct adapters of a tile are taken in
// turn.  One MFMA covers the 16 rows of a tile, so an adapter's A and B are read
// once for all its rows there; rows of other adapters enter as zeros (their x is not
// fetched) and their results are not stored.  First product: h^T = A x^T, rank by
// rows, K divided among the waves, whose sums are added in LDS in wave order.
// Second: y^T = B h^T, 64 columns of y at a time, so that a lane ends up with 16
// consecutive columns of its row.
#include <math.h>

#include "w8a8_common.h"
#include "../../include/lora.h"

using namespace w4k;

namespace {

constexpr int kRows = 16;              // rows of a tile
constexpr int kMaxR = 256;
constexpr int kMaxWaves = 8;
constexpr int kGroup = 64;             // columns that a wave takes at a time
constexpr int kUnit = 64;              // k that a wave takes at a time: a line of each row
constexpr uint32_t kNowhere = 0xf0000000u;   // past every buffer's end, with room for a row's offsets

struct LoraArgs {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const int* ranks;
    const float* scales;
    const int* adapter;
    const void* base;
    void* y;
    float* h;             // [slice][M][parts R], partial sums of the first product
    long long ldx, ldy;
    int y_dtype;
    int n, M, N, K, R, parts;
    int part_start[LORA_MAX_PARTS + 1];
    int block_start[LORA_MAX_PARTS + 1];   // first column block of each part
    int cols;             // columns of a block, a multiple of 64
    int turns;            // workgroups that share a tile's adapters
    int slices;           // slices of K (1 where the products are one launch)
};

template <bool BF16>
__device__ __forceinline__ float4_t mfma(const u32x4_t& a, const u32x4_t& b, const float4_t& c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(bitcast<bf16x8_t>(a), bitcast<bf16x8_t>(b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(bitcast<half8_t>(a), bitcast<half8_t>(b), c, 0, 0, 0);
}

// A tile's rows that share one adapter.
struct Rows {
    int m0;          // the tile's first row
    int id;          // adapter, -1: none
    int rank;        // rounded up to a multiple of 8
    uint32_t members;
};

// 16 RK ranks (from r0 on) of h for units [u0, u1) of this wave: acc[t][i] of lane (c, g)
// is rank r0 + 16 t + 4 g + i of row c.
template <bool BF16, int RK>
__device__ __forceinline__ void first_product(const LoraArgs& a, const Rows& r, int part, int r0, int u0, int u1, float4_t* acc) {
    constexpr int D = RK == 1 ? 6 : RK == 2 ? 4 : 3;   // units under way
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = 2u * a.K;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.a + ((size_t)r.id * a.parts + part) * a.R * a.K, (uint32_t)r.rank * row_bytes);
    const int last = min(kRows, a.M - r.m0) - 1;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)r.m0 * a.ldx, (uint32_t)(last * a.ldx + a.K) * 2u);
    const uint32_t x_row = (r.members >> c) & 1u ? (uint32_t)(c * a.ldx * 2) : kNowhere;
    const uint32_t a_row = (uint32_t)(r0 + c) * row_bytes;   // past the rank: past the buffer
    const uint32_t end = 2u * min(a.K, u1 * kUnit);
    u32x4_t xs[D][2], as[D][2][RK];
    auto load = [&](int i, int u) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t at = 2u * (u * kUnit) + 64 * s + 16 * g;
            xs[i][s] = bitcast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(rx, at < end ? x_row + at : kNowhere, 0, 0));
#pragma unroll
            for (int t = 0; t < RK; ++t)
                as[i][s][t] = bitcast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(ra, at < end ? a_row + 16 * t * row_bytes + at : kNowhere, 0, 0));
        }
    };
#pragma unroll
    for (int i = 0; i < D; ++i) load(i, u0 + i);
#pragma unroll 1
    for (int u = u0; u < u1; u += D) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < RK; ++t) acc[t] = mfma<BF16>(as[i][s][t], xs[i][s], acc[t]);
            load(i, u + i + D);
        }
    }
}

// The sums over units [u0, u1) and all ranks of a tile's rows into hf [16][R + 4],
// the waves' parts added in wave order.  part_lds: waves x RK KiB.
template <bool BF16, int RK>
__device__ __forceinline__ void sum_h(const LoraArgs& a, const Rows& r, int part, int u0, int u1, float* part_lds, float* hf) {
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), waves = blockDim.x >> 6;
    const int w0 = u0 + (u1 - u0) * wave / waves, w1 = u0 + (u1 - u0) * (wave + 1) / waves;
    for (int r0 = 0; r0 < r.rank; r0 += 16 * RK) {
        float4_t acc[RK];
#pragma unroll
        for (int i = 0; i < RK; ++i) acc[i] = float4_t{0.f, 0.f, 0.f, 0.f};
        first_product<BF16, RK>(a, r, part, r0, w0, w1, acc);
#pragma unroll
        for (int i = 0; i < RK; ++i) *(float4_t*)(part_lds + ((wave * RK + i) * 64 + lane) * 4) = acc[i];
        __syncthreads();
        for (int e = t; e < RK * 64; e += blockDim.x) {
            float4_t v = *(const float4_t*)(part_lds + e * 4);
            for (int w = 1; w < waves; ++w) v += *(const float4_t*)(part_lds + (w * RK * 64 + e) * 4);
            const int j = r0 + 16 * (e >> 6) + 4 * ((e >> 4) & 3);
            if (j < a.R) *(float4_t*)(hf + (e & 15) * (a.R + 4) + j) = v;
        }
        __syncthreads();
    }
}

__device__ __forceinline__ bool finite(float v) { return (bitcast<uint32_t>(v) & 0x7f800000u) != 0x7f800000u; }

// s h in NT terms of the dtype: hb [term][16][stride], ranks past the adapter's are zeros.
// fp16 has neither fp32's range nor a third term's use: each row is taken times a
// power of two that brings its largest element to 2^13, and back[] takes it back.
template <bool BF16, int NT>
__device__ __forceinline__ void split_h(const LoraArgs& a, const Rows& r, const float* hf, uint16_t* hb, int stride, float* back) {
    const int row = threadIdx.x >> 4, l = threadIdx.x & 15;
    if (row < kRows) {
        const float scale = r.id >= 0 && a.scales ? a.scales[r.id] : 1.f;
        const float* const src = hf + row * (a.R + 4);
        float up = 1.f;
        if constexpr (!BF16) {
            uint32_t top = 0;
            for (int j = l; j < r.rank; j += 16) {
                const float v = src[j] * scale;
                top = max(top, finite(v) ? bitcast<uint32_t>(v) & 0x7fffffffu : 0u);
            }
            top = max(top, dpp<0xB1>(top));
            top = max(top, dpp<0x4E>(top));
            top = max(top, dpp<0x141>(top));
            top = max(top, dpp<0x140>(top));
            const int e = max((int)(top >> 23), 40);                         // biased; below 2^-87 all the same
            up = bitcast<float>((uint32_t)(127 + 127 + 13 - e) << 23);      // 2^(13 - (e - 127)); e <= 254: at least 2^-114
            if (l == 0) back[row] = bitcast<float>((uint32_t)(e - 13) << 23);
        }
        for (int j = 2 * l; j < stride - 8; j += 32) {
            float v[2];
            uint32_t term[NT];
#pragma unroll
            for (int e = 0; e < 2; ++e) v[e] = j + e < r.rank ? src[j + e] * scale * up : 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // bf16 terms are cut off (a finite value stays finite), the last one is rounded.
                if constexpr (BF16)
                    term[n] = n == NT - 1 ? pk_bf16(v[0], v[1]) : (bitcast<uint32_t>(v[0]) >> 16) | (bitcast<uint32_t>(v[1]) & 0xffff0000u);
                else
                    term[n] = pk_f16(v[0], v[1]);
                const float t0 = BF16 ? bitcast<float>(term[n] << 16) : f16_bits_to_f32((uint16_t)term[n]);
                const float t1 = BF16 ? bitcast<float>(term[n] & 0xffff0000u) : f16_bits_to_f32((uint16_t)(term[n] >> 16));
                v[0] = finite(t0) ? v[0] - t0 : 0.f, v[1] = finite(t1) ? v[1] - t1 : 0.f;
                *(uint32_t*)(hb + (n * kRows + row) * stride + j) = term[n];
            }
        }
    }
    __syncthreads();
}

// y of columns [n0, n1) of a tile's rows.
template <bool BF16, int NT>
__device__ __forceinline__ void second_product(const LoraArgs& a, const Rows& r, int n0, int n1, const uint16_t* hb, int stride, const float* back) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int c = lane & 15, g = lane >> 4, steps = (r.rank + 31) / 32;
    const bool mine = (r.members >> c) & 1u;
    const float f = BF16 ? 1.f : back[c];
    const size_t row = (size_t)(r.m0 + c) * a.ldy;
    const uint32_t row_bytes = 2u * a.R;
    // Row 4 q + e of operand tile t is column 16 q + 4 t + e of the group.
    const uint32_t b_row = (16 * (c >> 2) + (c & 3)) * row_bytes;
    for (int n = n0 + kGroup * wave; n < n1; n += kGroup * waves) {
        const int col = n + 16 * g;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        if (a.base && mine) {
            if (col < n1) load8(a.base, a.y_dtype, row + col, v);
            if (col + 8 < n1) load8(a.base, a.y_dtype, row + col + 8, v + 8);
        }
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.b + ((size_t)max(r.id, 0) * a.N + n) * a.R, (uint32_t)min(kGroup, n1 - n) * row_bytes);
        float4_t acc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < steps; ++s) {
            const int j = 32 * s + 8 * g;
            u32x4_t w[4], h[NT];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                w[t] = bitcast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(rb, j < r.rank ? b_row + 4 * t * row_bytes + 2 * j : kNowhere, 0, 0));
#pragma unroll
            for (int i = 0; i < NT; ++i) h[i] = *(const u32x4_t*)(hb + (i * kRows + c) * stride + j);
#pragma unroll
            for (int i = NT - 1; i >= 0; --i)
#pragma unroll
                for (int t = 0; t < 4; ++t) acc[t] = mfma<BF16>(w[t], h[i], acc[t]);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __builtin_fmaf(acc[e >> 2][e & 3], f, v[e]);
        if (mine) {
            if (col < n1) store8(a.y, a.y_dtype, row + col, v);
            if (col + 8 < n1) store8(a.y, a.y_dtype, row + col + 8, v + 8);
        }
    }
}

// Calls f for this workgroup's share of the distinct adapters of a tile.
template <typename F>
__device__ __forceinline__ void each_adapter(const LoraArgs& a, int tile, int turn, bool with_none, F f) {
    const int lane = threadIdx.x & 63, m0 = tile * kRows;
    const bool there = lane < kRows && m0 + lane < a.M;
    int id = there ? a.adapter[m0 + lane] : -1;
    id = id < 0 || id >= a.n ? -1 : id;
    uint64_t left = __builtin_amdgcn_ballot_w64(there && (id >= 0 || with_none));
    for (int i = 0; left; ++i) {
        const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t same = __builtin_amdgcn_ballot_w64(there && id == one);
        left &= ~same;
        if (i % a.turns != turn) continue;
        Rows r{m0, one, 0, (uint32_t)same};
        if (one >= 0) {
            r.rank = a.ranks ? min(max(__builtin_amdgcn_readfirstlane(a.ranks[one]), 0), a.R) : a.R;
            r.rank = (r.rank + 7) & ~7;
        }
        f(r);
    }
}

enum Mode { kBoth, kFirst, kSecond };

// MODE kBoth: both products in one launch, a workgroup for (tile, turn, column block); the
// first product is made again by each block of columns, from L2.  Where that
// costs more than a second launch, kFirst makes slices of the sums over K and
// kSecond adds them in slice order.
template <bool BF16, int NT, int RK, Mode MODE>
__global__ __launch_bounds__(kMaxWaves * 64) void lora_kernel(LoraArgs a) {
    extern __shared__ __attribute__((aligned(16))) float smem[];
    const int t = threadIdx.x;
    const int stride = (a.R + 31) / 32 * 32 + 8;                   // of a row of hb, in elements
    float* const back = smem;                                      // [16]
    float* const hf = smem + kRows;                                // [16][R + 4]
    float* const scratch = hf + kRows * (a.R + 4);                 // the waves' sums, then hb
    uint16_t* const hb = (uint16_t*)scratch;
    const int blocks = a.block_start[a.parts];
    if constexpr (MODE == kFirst) {
        const int slice = blockIdx.x % a.slices, part = blockIdx.x / a.slices % a.parts;
        const uint32_t unit = blockIdx.x / ((uint32_t)a.slices * a.parts);
        const int turn = unit % a.turns, tile = unit / a.turns;
        const int units = (a.K + kUnit - 1) / kUnit;
        const int u0 = (long long)units * slice / a.slices, u1 = (long long)units * (slice + 1) / a.slices;
        each_adapter(a, tile, turn, false, [&](const Rows& r) {
            sum_h<BF16, RK>(a, r, part, u0, u1, scratch, hf);
            float* const dst = a.h + ((size_t)slice * a.M + r.m0) * a.parts * a.R + part * a.R;
            for (int e = t; e < kRows * (r.rank / 4); e += blockDim.x) {
                const int row = e / (r.rank / 4), j = e % (r.rank / 4) * 4;
                if ((r.members >> row) & 1u) *(float4_t*)(dst + (size_t)row * a.parts * a.R + j) = *(const float4_t*)(hf + row * (a.R + 4) + j);
            }
            __syncthreads();
        });
    } else {
        const int block = blockIdx.x % (uint32_t)blocks;
        const uint32_t unit = blockIdx.x / (uint32_t)blocks;
        const int turn = unit % a.turns, tile = unit / a.turns;
        int part = 0;
        while (part + 1 < a.parts && block >= a.block_start[part + 1]) ++part;
        const int n0 = a.part_start[part] + (block - a.block_start[part]) * a.cols, n1 = min(n0 + a.cols, a.part_start[part + 1]);
        // base copied for rows without an adapter, unless it is y itself
        each_adapter(a, tile, turn, a.base != a.y, [&](const Rows& r) {
            if constexpr (MODE == kBoth) {
                sum_h<BF16, RK>(a, r, part, 0, (a.K + kUnit - 1) / kUnit, scratch, hf);
            } else {
                const float* const src = a.h + (size_t)r.m0 * a.parts * a.R + part * a.R;
                for (int e = t; e < kRows * (r.rank / 4); e += blockDim.x) {
                    const int row = e / (r.rank / 4), j = e % (r.rank / 4) * 4;
                    float4_t v = {0.f, 0.f, 0.f, 0.f};
                    if ((r.members >> row) & 1u)
                        for (int s = 0; s < a.slices; ++s) v += *(const float4_t*)(src + ((size_t)s * a.M + row) * a.parts * a.R + j);
                    *(float4_t*)(hf + row * (a.R + 4) + j) = v;
                }
                __syncthreads();
            }
            split_h<BF16, NT>(a, r, hf, hb, stride, back);
            second_product<BF16, NT>(a, r, n0, n1, hb, stride, back);
            __syncthreads();
        });
    }
}

typedef void (*kernel_t)(LoraArgs);

template <bool BF16, int NT, int RK>
kernel_t pick(Mode m) {
    return m == kBoth ? lora_kernel<BF16, NT, RK, kBoth> : m == kFirst ? lora_kernel<BF16, NT, RK, kFirst> : lora_kernel<BF16, NT, RK, kSecond>;
}
template <bool BF16, int NT>
kernel_t pick(int rk, Mode m) {
    return rk == 1 ? pick<BF16, NT, 1>(m) : rk == 2 ? pick<BF16, NT, 2>(m) : pick<BF16, NT, 4>(m);
}

struct Plan {
    bool split;           // two launches
    int rk;               // rank tiles that a wave takes at once
    int threads, turns, cols, slices;
    long long tiles;
    size_t ws;
};

Plan make_plan(int M, int N, int K, int R, int parts) {
    Plan p{};
    const long long cus = w4h::cu_count();
    p.tiles = (M + kRows - 1) / kRows;
    p.rk = R <= 16 ? 1 : R <= 32 ? 2 : 4;
    p.turns = M <= 512 ? (M < kRows ? M : kRows) : 1;
    const long long units = M <= 512 ? M : p.tiles;      // (tile, adapter) pairs at most, or about
    p.split = (long long)R * K > 200000;
    p.threads = 512;
    // Columns of a block: enough blocks for two workgroups per CU, 64 columns per wave at least.
    const long long want = (2 * cus + units - 1) / units;
    long long cols = (N + want - 1) / want;
    cols = (cols + kGroup - 1) / kGroup * kGroup;
    const long long least = p.split ? 4 * kGroup : 2 * kGroup;
    p.cols = (int)(cols < least ? least : cols);
    p.slices = 1;
    if (p.split) {
        const long long k_units = (K + kUnit - 1) / kUnit;
        long long s = (2 * cus + units * parts - 1) / (units * parts);
        s = s < k_units / 8 ? s : k_units / 8;            // a unit for each wave at least
        s = s < 32 ? s : 32;
        p.slices = (int)(s < 1 ? 1 : s);
        p.ws = w4h::ws_bytes((size_t)p.slices * M * parts * R * sizeof(float));
    }
    return p;
}

size_t lds_bytes(const Plan& p, int R, int terms, Mode m) {
    const size_t sums = (size_t)(p.threads / 64) * p.rk * 1024, hb = (size_t)terms * kRows * ((R + 31) / 32 * 32 + 8) * 2;
    const size_t rest = m == kFirst ? sums : m == kSecond || hb > sums ? hb : sums;
    return (kRows + (size_t)kRows * (R + 4)) * sizeof(float) + rest;
}

int check_shape(int M, int N, int K, int R, int parts) {
    if (M < 1 || M > (1 << 26) || N < 8 || N > (1 << 24) || N % 8 || K < 8 || K > (1 << 20) || K % 8 || R < 8 || R > kMaxR || R % 8 ||
        parts < 1 || parts > LORA_MAX_PARTS)
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

// Workgroups of the launches that a plan makes, the columns' blocks of each part at most one more than its share.
bool fits(const Plan& p, int N, int parts) {
    const long long blocks = (N + p.cols - 1) / p.cols + parts, units = p.tiles * p.turns;
    return units * blocks * p.threads <= kMaxLanes && units * parts * p.slices * p.threads <= kMaxLanes;
}

}  // namespace

extern "C" int lora_workspace_bytes(int M, int N, int K, int R, int parts, size_t* bytes) {
    if (!bytes) return W4A16_ERR_NULL;
    if (int rc = check_shape(M, N, K, R, parts)) return rc;
    const Plan p = make_plan(M, N, K, R, parts);
    if (!fits(p, N, parts)) return W4A16_ERR_UNSUPPORTED;
    *bytes = p.ws;
    return W4A16_OK;
}

extern "C" int lora_add(const void* x, int dtype, long long ldx, const void* a, const void* b, const int32_t* ranks,
                        const float* scales, int n_adapters, const int32_t* adapter, const void* base, void* y,
                        int y_dtype, long long ldy, const int* part_cols, int parts, int M, int N, int K, int R,
                        void* workspace, size_t workspace_bytes, w4a16_stream_t stream) {
    if (!x || !a || !b || !adapter || !y) return W4A16_ERR_NULL;
    if (dtype != W4A16_F16 && dtype != W4A16_BF16) return W4A16_ERR_DTYPE;
    if (y_dtype != W4A16_F32 && y_dtype != W4A16_F16 && y_dtype != W4A16_BF16) return W4A16_ERR_DTYPE;
    if (int rc = check_shape(M, N, K, R, parts)) return rc;
    if (n_adapters < 1 || ldx < K || ldx % 8 || ldx >= (1 << 26) || ldy < N || ldy % 8) return W4A16_ERR_SHAPE;
    if (parts > 1 && !part_cols) return W4A16_ERR_NULL;
    LoraArgs g{};
    for (int i = 0; i < parts; ++i) {
        const int cols = parts == 1 && !part_cols ? N : part_cols[i];
        if (cols < 8 || cols > N - g.part_start[i] || (i + 1 < parts && cols % kGroup)) return W4A16_ERR_SHAPE;
        g.part_start[i + 1] = g.part_start[i] + cols;
    }
    if (g.part_start[parts] != N) return W4A16_ERR_SHAPE;
    for (const void* p : {x, a, b, base, (const void*)y, (const void*)workspace})
        if (!w4h::aligned16(p)) return W4A16_ERR_ALIGN;
    if (((uintptr_t)ranks & 3) || ((uintptr_t)scales & 3) || ((uintptr_t)adapter & 3)) return W4A16_ERR_ALIGN;
    const Plan p = make_plan(M, N, K, R, parts);
    if (!fits(p, N, parts)) return W4A16_ERR_UNSUPPORTED;
    if (p.ws && !workspace) return W4A16_ERR_NULL;
    if (workspace_bytes < p.ws) return W4A16_ERR_WORKSPACE;
    g.x = (const uint16_t*)x, g.a = (const uint16_t*)a, g.b = (const uint16_t*)b;
    g.ranks = ranks, g.scales = scales, g.adapter = adapter, g.base = base, g.y = y, g.h = (float*)w4h::ws_part(workspace);
    g.ldx = ldx, g.ldy = ldy, g.y_dtype = y_dtype;
    g.n = n_adapters, g.M = M, g.N = N, g.K = K, g.R = R, g.parts = parts;
    g.cols = p.cols, g.turns = p.turns, g.slices = p.slices;
    for (int i = 0; i < parts; ++i) {
        const int cols = g.part_start[i + 1] - g.part_start[i];
        g.block_start[i + 1] = g.block_start[i] + (cols + p.cols - 1) / p.cols;
    }
    const bool bf16 = dtype == W4A16_BF16;
    const int terms = bf16 && y_dtype == W4A16_F32 ? 3 : 2;
    auto kernel = [&](Mode m) {
        return !bf16 ? pick<false, 2>(p.rk, m) : terms == 2 ? pick<true, 2>(p.rk, m) : pick<true, 3>(p.rk, m);
    };
    const long long units = p.tiles * p.turns;
    const hipStream_t st = (hipStream_t)stream;
    w4h::begin_launches();
    if (p.split)
        hipLaunchKernelGGL(kernel(kFirst), dim3((unsigned)(units * parts * p.slices)), dim3(p.threads), lds_bytes(p, R, terms, kFirst), st, g);
    const Mode m = p.split ? kSecond : kBoth;
    hipLaunchKernelGGL(kernel(m), dim3((unsigned)(units * g.block_start[parts])), dim3(p.threads), lds_bytes(p, R, terms, m), st, g);
    w4h::note_variant("%s launches=%lld ranks=%lld threads=%lld turns=%lld cols=%lld slices=%lld", "lora", p.split ? 2 : 1, 16 * p.rk, p.threads,
                      p.turns, p.cols, p.slices);
    return w4h::launch_status();
}
