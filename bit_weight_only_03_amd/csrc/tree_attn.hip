// tree_attn.hip -- attention of a tree of drafted tokens over a paged cache.
//
// One pass over the cache with the running maximum and sum of a softmax.  The
// T G rows (drafts x query heads of one kv head) of a request share its keys,
// so a workgroup takes a kv head, up to 16 RT WR rows and a range of keys; its
// WK x WR waves are WK groups that take tiles of 32 keys in turn and, within a
// group, WR waves with RT operand tiles of 16 rows each.
//
// Products.  Scores are computed transposed, S^T = K Q^T, so that a lane holds
// one row's scores at keys 4g .. 4g+3 of each 16 (g = lane / 16): exactly the
// layout in which the product O^T = V^T P^T takes P as its B operand once the
// 32 slots of k are named (g, i) -> key 4g + i (i < 4), 16 + 4g + i - 4.  The
// probabilities never leave the lane, and neither do the row's maximum, sum
// and rescaling factor.  V^T as the A operand needs eight keys of one column d
// per lane; the columns of an operand tile are free, so lane r of tile t takes
// column (D/16) r + t: it loads D/16 consecutive columns of each key and pairs
// them up with one byte permute per register.
//
// Tiles of K and V go from the cache straight to LDS, whole rows of a page, two
// tiles deep per group.  K's 16-byte chunks are permuted with the key on the
// way, so that reading one chunk of 16 keys is free of bank conflicts.
#include <atomic>

#include "w8a8_common.h"
#include "../../include/tree_attn.h"

using namespace w4k;

namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef const __attribute__((address_space(1))) void* global_ptr_t;

constexpr int kTile = 32;              // keys per tile
constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kLn2 = 0x1.62e43p-1f;
constexpr int kMaxSplit = 64;
constexpr int kMaxDevices = 64;
constexpr int kMaxDynamicLds = 160 * 1024;

struct TreeArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int* table;
    const int* lens;
    const uint64_t* mask;
    void* out;
    float* lse;
    float* part_o;     // [unit][row][split][D] sums that are not divided yet
    float2* part_ml;   // [unit][row][split] maximum (log2 units) and sum
    long long q_stride, page_stride, token_stride, head_stride;
    int num_pages, page_shift, table_stride;
    int max_len;
    float scale2;      // scale * log2(e)
    int B, T, Hq, Hkv, G, R;
    int S, RB;         // splits of the keys, blocks of rows
};

template <bool BF16>
__device__ __forceinline__ float4_t mfma(const u32x4_t& a, const u32x4_t& b, const float4_t& c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(bitcast<bf16x8_t>(a), bitcast<bf16x8_t>(b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(bitcast<half8_t>(a), bitcast<half8_t>(b), c, 0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return BF16 ? pk_bf16(a, b) : pk_f16(a, b);
}

template <bool BF16>
__device__ __forceinline__ float unpack1(uint32_t h) {   // the low 16 bits
    return BF16 ? bitcast<float>(h << 16) : f16_bits_to_f32((uint16_t)h);
}

template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t h) {
    constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
    return (h & kExp) == kExp;
}

// The largest (sum) over the four lanes that hold one row, 16 apart.
__device__ __forceinline__ float max4(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(bitcast<uint32_t>(x), bitcast<uint32_t>(x), false, false);
    x = __builtin_fmaxf(bitcast<float>((uint32_t)a[0]), bitcast<float>((uint32_t)a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(bitcast<uint32_t>(x), bitcast<uint32_t>(x), false, false);
    return __builtin_fmaxf(bitcast<float>((uint32_t)b[0]), bitcast<float>((uint32_t)b[1]));
}
__device__ __forceinline__ float sum4(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(bitcast<uint32_t>(x), bitcast<uint32_t>(x), false, false);
    x = bitcast<float>((uint32_t)a[0]) + bitcast<float>((uint32_t)a[1]);
    auto b = __builtin_amdgcn_permlane16_swap(bitcast<uint32_t>(x), bitcast<uint32_t>(x), false, false);
    return bitcast<float>((uint32_t)b[0]) + bitcast<float>((uint32_t)b[1]);
}

// Probabilities are taken as 2^(x - m + kLift).  In f16 that keeps them normal
// down to 2^-29 of the largest: without it the many small ones of a long
// context (below 2^-14) would be rounded to f16's subnormal grid, all the same
// way, and 150 000 of them add up to a visible share.  The sum carries the
// same factor, so only lse takes it back.  bf16 has fp32's exponents.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 15.f;

// 2^(m - top), 0 for a part that has seen nothing (m = -inf).
__device__ __forceinline__ float weight_of(float m, float top) {
    return m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - top);
}

// The address of a row's result, or null past the rows.
__device__ __forceinline__ size_t out_row(const TreeArgs& a, int b, int kvh, int row) {
    return ((size_t)b * a.T + row / a.G) * a.Hq + kvh * a.G + row % a.G;
}

template <bool BF16, int D, int RT, int WK, int WR>
__global__ __launch_bounds__(WK* WR * 64) void tree_attn_kernel(TreeArgs a) {
    constexpr int DT = D / 16;                 // operand tiles of O^T
    constexpr int KS = D / 32;                 // products per score tile
    constexpr int kChunks = D / 8;             // 16-byte chunks of a key
    constexpr int kSwz = kChunks < 16 ? kChunks - 1 : 15;
    constexpr int kHalf = kTile * D * 2;       // bytes of a tile of K or of V
    constexpr int kStage = 2 * kHalf;
    constexpr int kKeys = 512 / D;             // keys per load instruction
    constexpr int kPer = kTile / kKeys / WR;   // loads of K (and of V) per wave and tile
    constexpr int kRows = 16 * RT * WR;
    constexpr int kAux = WR < 4 ? kAuxNT : 0;  // few rows: read once; more: other blocks of rows read it again
    static_assert(kPer >= 1, "a wave loads whole instructions");
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63;
    const int kg = wave / WR, wr = wave % WR, c = lane & 15, g = lane >> 4;

    // Consecutive workgroups go to the XCDs in turn: the blocks of rows that
    // read the same keys sit 8 apart, on one XCD.
    const int u8 = blockIdx.x >> 3, rb = u8 % a.RB, id = (u8 / a.RB) * 8 + (blockIdx.x & 7);
    if (id >= a.B * a.Hkv * a.S) return;
    const int split = id % a.S, unit = id / a.S, kvh = unit % a.Hkv, b = unit / a.Hkv;
    const int len = min(max(a.lens[b], 0), a.max_len), total = len + a.T;
    const int tiles = (total + kTile - 1) / kTile;
    const int t0 = (int)((long long)tiles * split / a.S), t1 = (int)((long long)tiles * (split + 1) / a.S);
    const int nt = t1 - t0 > kg ? (t1 - t0 - kg + WK - 1) / WK : 0;   // this group's tiles
    const int loops = (t1 - t0 + WK - 1) / WK;                        // the same for every group (barriers)

    const int* const table = a.table + (size_t)b * a.table_stride;
    const long long head = kvh * a.head_stride;
    uint8_t* const ring = smem + kg * 2 * kStage;
    const int key_in = lane / kChunks, pos = lane % kChunks;

    // Lane j of 32: the page of key j of the group's tile n (the last key's
    // page past the end).
    auto page_of = [&](int n) {
        const int p = min((t0 + kg + n * WK) * kTile + (lane & 31), total - 1);
        return min(max(table[p >> a.page_shift], 0), a.num_pages - 1);
    };
    auto issue = [&](int n, int pages) {
        uint8_t* const to = ring + (n & 1) * kStage;
        const int first = (t0 + kg + n * WK) * kTile;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = (wr * kPer + i) * kKeys + key_in;      // key of the tile
            const int p = min(first + j, total - 1);
            const long long row = (long long)__shfl(pages, j) * a.page_stride +
                                  (long long)(p & ((1 << a.page_shift) - 1)) * a.token_stride + head;
            const uint16_t* const kp = a.k + row + 8 * (pos ^ (j & kSwz));
            const uint16_t* const vp = a.v + row + 8 * pos;
            uint8_t* const at = to + (wr * kPer + i) * 1024;
            __builtin_amdgcn_global_load_lds((global_ptr_t)kp, (lds_ptr_t)at, 16, 0, kAux);
            __builtin_amdgcn_global_load_lds((global_ptr_t)vp, (lds_ptr_t)(at + kHalf), 16, 0, kAux);
        }
    };

    // The rows: B operand of the scores, and each row's mask.
    const int row0 = rb * kRows + wr * RT * 16;
    u32x4_t qf[RT][KS];
    uint64_t see[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = row0 + 16 * rt + c;
        const bool there = row < a.R;
        const int tok = there ? row / a.G : 0;
        see[rt] = there ? a.mask[(size_t)b * a.T + tok] : 0;
        const uint16_t* const qp = a.q + ((size_t)b * a.T + tok) * a.q_stride + (size_t)(kvh * a.G + (there ? row % a.G : 0)) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[rt][s] = there ? *(const u32x4_t*)(qp + 32 * s + 8 * g) : u32x4_t{0, 0, 0, 0};
    }
    float4_t o[RT][DT];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -__builtin_inff(), l[rt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[rt][d] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    int pages = 0;   // of the tile that is issued next
    if (nt > 0) {
        const int pages0 = page_of(0);
        pages = page_of(min(1, nt - 1));
        issue(0, pages0);
    }
    for (int n = 0; n < loops; ++n) {
        const bool live = n < nt;
        if constexpr (WR == 1) {
            if (!live) break;
        }
        // The next tile's loads go out before this one is waited for (one wave
        // to a group: the other buffer is its own and read), or after the
        // barrier that says the other buffer is read.  The page numbers of the
        // tile after it are asked for before them, so that waiting for the
        // numbers never waits for these loads.  Past the last tile the last one
        // is loaded again, which nothing reads.
        const int after = min(n + 1, nt - 1);
        if constexpr (WR == 1) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            const int next = page_of(min(n + 2, nt - 1));
            __builtin_amdgcn_sched_barrier(0);
            if (after > n) issue(after, pages);
            __builtin_amdgcn_sched_barrier(0);
            pages = next;
            if (after > n)
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kPer) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (live && after > n) {
                const int next = page_of(min(n + 2, nt - 1));
                issue(after, pages);
                pages = next;
            }
            if (!live) continue;
        }
        const uint8_t* const kt = ring + (n & 1) * kStage;
        const uint8_t* const vt = kt + kHalf;
        const int first = (t0 + kg + n * WK) * kTile;
        const bool edge = first + kTile > len;   // drafts or the end inside (the same for the whole wave)

        float4_t sc[2][RT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) sc[h][rt] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const u32x4_t kf = *(const u32x4_t*)(kt + (16 * h + c) * D * 2 + 16 * ((4 * s + g) ^ (c & kSwz)));
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) sc[h][rt] = mfma<BF16>(kf, qf[rt][s], sc[h][rt]);
            }
        }
        u32x4_t pf[RT];   // probabilities: the B operand of the product with V
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][rt][i & 3] * a.scale2;
            if (edge) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int p = first + 16 * (i >> 2) + 4 * g + (i & 3), j = p - len;
                    const bool sees = j < 0 || (j < a.T && ((see[rt] >> (j & 63)) & 1));
                    x[i] = sees ? x[i] : -__builtin_inff();
                }
            }
            float top = x[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, x[i]);
            top = max4(top);
            const float mn = __builtin_fmaxf(m[rt], top);
            if (__builtin_amdgcn_ballot_w64(mn > m[rt])) {   // some row's maximum rose
                const float f = weight_of(m[rt], mn);
                l[rt] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[rt][d][q] *= f;
                m[rt] = mn;
            }
            const float base = mn == -__builtin_inff() ? 0.f : mn - kLift<BF16>;   // nothing seen yet: every p is 2^-inf = 0
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = __builtin_amdgcn_exp2f(x[i] - base);
                sum += x[i];
            }
            l[rt] += sum;   // this lane's keys; the four lanes of a row are added at the end
#pragma unroll
            for (int j = 0; j < 4; ++j) pf[rt][j] = pack2<BF16>(x[2 * j], x[2 * j + 1]);
        }
        // V: D/16 columns of this lane's eight keys.
        constexpr int VW = D / 32;   // dwords of a key per lane
        uint32_t vr[8][VW];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t* const p = vt + (16 * (i >> 2) + 4 * g + (i & 3)) * D * 2 + c * VW * 4;
            if constexpr (VW == 2) {
                const u32x2_t v = *(const u32x2_t*)p;
                vr[i][0] = v[0], vr[i][1] = v[1];
            } else {
#pragma unroll
                for (int w = 0; w < VW; w += 4) {
                    const u32x4_t v = *(const u32x4_t*)(p + 4 * w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) vr[i][w + e] = v[e];
                }
            }
        }
        if (edge) {
            // Keys past the end count as zeros.  A draft's infinity or NaN must
            // not reach the rows that do not see it (0 * inf): it is taken out
            // of the product and added, key by key, to the rows that do.
            uint64_t odd[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = first + 16 * (i >> 2) + 4 * g + (i & 3);
                bool bad = false;
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    const uint32_t v = p < total ? vr[i][w] : 0u;
                    const bool lo = not_finite<BF16>(v), hi = not_finite<BF16>(v >> 16);
                    bad |= p >= len && (lo || hi);
                    vr[i][w] = p < len ? v : (lo ? 0u : v & 0xffffu) | (hi ? 0u : v & 0xffff0000u);
                }
                odd[i] = __builtin_amdgcn_ballot_w64(bad);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                for (int gk = 0; gk < 4 && odd[i]; ++gk) {
                    if (!((odd[i] >> (16 * gk)) & 0xffff)) continue;
                    const int j = 16 * (i >> 2) + 4 * gk + (i & 3), draft = first + j - len;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const uint32_t pw = __shfl(pf[rt][i >> 1], 16 * gk + c);
                        const float p = unpack1<BF16>(i & 1 ? pw >> 16 : pw & 0xffffu);
                        const bool sees = (see[rt] >> (draft & 63)) & 1;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int d = 0; d < DT; ++d) {
                                const uint32_t h = *(const uint16_t*)(vt + j * D * 2 + (DT * (4 * g + q) + d) * 2);
                                if (sees && not_finite<BF16>(h)) o[rt][d][q] += p * unpack1<BF16>(h);
                            }
                    }
                }
            }
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            u32x4_t va;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                va[j] = __builtin_amdgcn_perm(vr[2 * j + 1][d >> 1], vr[2 * j][d >> 1], d & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) o[rt][d] = mfma<BF16>(va, pf[rt], o[rt][d]);
        }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();

    // The groups' parts, each a sum with its own maximum: [group][row of the block].
    float* const ml = (float*)smem;                                  // [WK][kRows][2]
    float* const os = (float*)(smem + WK * kRows * 2 * sizeof(float));   // [WK][kRows][D]
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] = sum4(l[rt]);
        if (g == 0) {
            float* const at = ml + (kg * kRows + wr * RT * 16 + 16 * rt + c) * 2;
            at[0] = m[rt], at[1] = l[rt];
        }
    }
    __syncthreads();
    const size_t first_row = (size_t)unit * a.R;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int in_block = wr * RT * 16 + 16 * rt + c, row = rb * kRows + in_block;
        float top = m[rt];
#pragma unroll
        for (int w = 0; w < WK; ++w) top = __builtin_fmaxf(top, ml[(w * kRows + in_block) * 2]);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const float* const at = ml + (w * kRows + in_block) * 2;
            sum += weight_of(at[0], top) * at[1];
        }
        float f = weight_of(m[rt], top);
        if (a.S == 1) f = sum == 0.f ? 0.f : f / sum;
        if (kg == 0 && g == 0 && row < a.R) {
            if (a.S > 1)
                a.part_ml[(first_row + row) * a.S + split] = float2{top, sum};
            else if (a.lse)
                a.lse[out_row(a, b, kvh, row)] = sum == 0.f ? -__builtin_inff() : (top - kLift<BF16> + __builtin_log2f(sum)) * kLn2;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int d = 0; d < DT; ++d) o[rt][d][q] *= f;
        // Lane c, g holds columns DT (4g + q) + d of its row.
        if constexpr (WK > 1) {
            float* const to = os + ((size_t)kg * kRows + in_block) * D;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int d = 0; d < DT; d += 4)
                    *(float4_t*)(to + DT * (4 * g + q) + d) = float4_t{o[rt][d][q], o[rt][d + 1][q], o[rt][d + 2][q], o[rt][d + 3][q]};
        } else if (row < a.R) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int d = 0; d < DT; d += 4) {
                    const int col = DT * (4 * g + q) + d;
                    if (a.S > 1)
                        *(float4_t*)(a.part_o + ((first_row + row) * a.S + split) * D + col) =
                            float4_t{o[rt][d][q], o[rt][d + 1][q], o[rt][d + 2][q], o[rt][d + 3][q]};
                    else
                        *(u32x2_t*)((uint16_t*)a.out + out_row(a, b, kvh, row) * D + col) =
                            u32x2_t{pack2<BF16>(o[rt][d][q], o[rt][d + 1][q]), pack2<BF16>(o[rt][d + 2][q], o[rt][d + 3][q])};
                }
        }
    }
    if constexpr (WK > 1) {
        __syncthreads();
        for (int e = t * 4; e < kRows * D; e += WK * WR * 256) {
            const int row = rb * kRows + e / D, col = e % D;
            if (row >= a.R) break;
            float4_t v = *(const float4_t*)(os + e);
#pragma unroll
            for (int w = 1; w < WK; ++w) v += *(const float4_t*)(os + (size_t)w * kRows * D + e);
            if (a.S > 1)
                *(float4_t*)(a.part_o + ((first_row + row) * a.S + split) * D + col) = v;
            else
                *(u32x2_t*)((uint16_t*)a.out + out_row(a, b, kvh, row) * D + col) =
                    u32x2_t{pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3])};
        }
    }
}

// Joins the S parts of each row: o = sum 2^(m_s - top) o_s / sum 2^(m_s - top) l_s,
// in order of s.  A wave per row: lane s holds part s's weight (S <= 64), then
// every lane D/64 columns.
template <bool BF16, int D>
__global__ __launch_bounds__(256) void tree_merge_kernel(TreeArgs a, long long rows) {
    constexpr int C = D / 64;
    const int lane = threadIdx.x & 63;
    const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= rows) return;
    const int unit = (int)(r / a.R), row = (int)(r % a.R);
    float2 ml = float2{-__builtin_inff(), 0.f};
    if (lane < a.S) ml = a.part_ml[r * a.S + lane];
    float top = ml.x;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, s));
    const float f = weight_of(ml.x, top);
    float sum = f * ml.y;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
    float v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = 0.f;
    const float* const src = a.part_o + r * a.S * D + lane * C;
    for (int s = 0; s < a.S; ++s) {
        const float w = __shfl(f, s);
        if (w == 0.f) continue;   // a part that saw nothing, or whose weight is 0
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = __builtin_fmaf(w, src[(size_t)s * D + i], v[i]);
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    const size_t at = out_row(a, unit / a.Hkv, unit % a.Hkv, row);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const uint32_t h = pack2<BF16>(v[i] * inv, 0.f);
        ((uint16_t*)a.out)[at * D + lane * C + i] = (uint16_t)h;
    }
    if (lane == 0 && a.lse) a.lse[at] = sum == 0.f ? -__builtin_inff() : (top - kLift<BF16> + __builtin_log2f(sum)) * kLn2;
}

typedef void (*kernel_t)(TreeArgs);

struct Plan {
    kernel_t kernel[2];   // f16, bf16
    int rows;             // rows of a workgroup
    int wk;               // key groups
    int threads;
    size_t lds;
    int S, RB;
    long long units;      // requests x kv heads
    size_t ws;
};

template <int D, int RT, int WK, int WR>
void use(Plan& p) {
    p.kernel[0] = tree_attn_kernel<false, D, RT, WK, WR>;
    p.kernel[1] = tree_attn_kernel<true, D, RT, WK, WR>;
    p.rows = 16 * RT * WR, p.wk = WK, p.threads = 64 * WK * WR;
    const size_t ring = (size_t)WK * 2 * 2 * kTile * D * 2;
    const size_t join = (size_t)WK * p.rows * (2 + (WK > 1 ? D : 0)) * sizeof(float);
    p.lds = ring > join ? ring : join;
}

template <int D>
void use_rows(Plan& p, int R) {
    if constexpr (D == 256) {
        if (R <= 16) use<D, 1, 2, 1>(p);
        else if (R <= 32) use<D, 1, 2, 2>(p);
        else use<D, 1, 1, 4>(p);
    } else {
        if (R <= 16) use<D, 1, 4, 1>(p);
        else if (R <= 32) use<D, 2, 4, 1>(p);
        else if (R <= 64) use<D, 2, 2, 2>(p);
        else use<D, 2, 1, 4>(p);
    }
}

Plan make_plan(int B, int T, int Hq, int Hkv, int D, int max_len) {
    Plan p{};
    const int R = T * (Hq / Hkv);
    if (D == 64) use_rows<64>(p, R);
    else if (D == 128) use_rows<128>(p, R);
    else use_rows<256>(p, R);
    p.RB = (R + p.rows - 1) / p.rows;
    p.units = (long long)B * Hkv;
    // One workgroup or more per CU, each group of waves with two tiles at least.
    const long long tiles = ((long long)max_len + T + kTile - 1) / kTile;
    const int per_cu = (int)(kMaxDynamicLds / p.lds) < 2 ? 1 : 2;
    long long S = (long long)w4h::cu_count() * per_cu / (p.units * p.RB);
    S = S < kMaxSplit ? S : kMaxSplit;
    S = S < tiles / (2 * p.wk) ? S : tiles / (2 * p.wk);
    p.S = S < 1 ? 1 : (int)S;
    p.ws = p.S > 1 ? w4h::ws_bytes((size_t)p.units * R * p.S * (D + 2) * sizeof(float)) : 0;
    return p;
}

// The kernels' dynamic LDS may pass the default limit: said once per process and device.
void allow_lds() {
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices || done[dev].load(std::memory_order_acquire)) return;
    for (int D : {64, 128, 256})
        for (int R : {1, 17, 33, 65}) {
            Plan q{};
            if (D == 64) use_rows<64>(q, R);
            else if (D == 128) use_rows<128>(q, R);
            else use_rows<256>(q, R);
            for (kernel_t k : q.kernel)
                (void)hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicLds);
        }
    done[dev].store(true, std::memory_order_release);
}

int check_shape(int B, int T, int Hq, int Hkv, int D, int max_len) {
    if (B < 1 || T < 1 || T > 64 || Hkv < 1 || Hq < Hkv || Hq % Hkv || max_len < 0 || max_len > (1 << 30))
        return W4A16_ERR_SHAPE;
    if (Hq > (1 << 16) || (long long)B * Hq > (1LL << 24)) return W4A16_ERR_SHAPE;
    if (D != 64 && D != 128 && D != 256) return W4A16_ERR_UNSUPPORTED;
    return W4A16_OK;
}

}  // namespace

extern "C" int tree_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int max_len, size_t* bytes) {
    if (!bytes) return W4A16_ERR_NULL;
    if (int rc = check_shape(B, T, Hq, Hkv, D, max_len)) return rc;
    *bytes = make_plan(B, T, Hq, Hkv, D, max_len).ws;
    return W4A16_OK;
}

extern "C" int tree_attn(const void* q, long long q_stride, const void* k, const void* v, int dtype,
                         int num_pages, int page_size, long long page_stride, long long token_stride,
                         long long head_stride, const int32_t* block_table, int table_stride,
                         const int32_t* lens, int max_len, const uint64_t* tree_mask, float scale, void* out,
                         float* lse, int B, int T, int Hq, int Hkv, int D, void* workspace,
                         size_t workspace_bytes, w4a16_stream_t stream) {
    if (!q || !k || !v || !block_table || !lens || !tree_mask || !out) return W4A16_ERR_NULL;
    if (dtype != W4A16_F16 && dtype != W4A16_BF16) return W4A16_ERR_DTYPE;
    if (int rc = check_shape(B, T, Hq, Hkv, D, max_len)) return rc;
    if (num_pages < 1 || page_size < 1 || (page_size & (page_size - 1)) || table_stride < 1 ||
        (long long)table_stride * page_size < (long long)max_len + T)
        return W4A16_ERR_SHAPE;
    if (q_stride < (long long)Hq * D || q_stride % 8 || page_stride < 0 || token_stride < 0 || head_stride < 0 ||
        page_stride % 8 || token_stride % 8 || head_stride % 8 || !(scale == scale) || scale - scale != 0.f)
        return W4A16_ERR_SHAPE;
    if (!w4h::aligned16(q) || !w4h::aligned16(k) || !w4h::aligned16(v) || !w4h::aligned16(out) ||
        !w4h::aligned16(workspace) || ((uintptr_t)lens & 3) || ((uintptr_t)block_table & 3) ||
        ((uintptr_t)tree_mask & 7) || ((uintptr_t)lse & 3))
        return W4A16_ERR_ALIGN;
    const Plan p = make_plan(B, T, Hq, Hkv, D, max_len);
    const long long blocks = (p.units * p.S + 7) / 8 * 8 * p.RB;
    const int R = T * (Hq / Hkv);
    const long long rows = p.units * R;
    if (blocks > 0x7fffffffLL) return W4A16_ERR_UNSUPPORTED;
    if (p.ws && !workspace) return W4A16_ERR_NULL;
    if (workspace_bytes < p.ws) return W4A16_ERR_WORKSPACE;
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    TreeArgs a{};
    a.q = (const uint16_t*)q, a.k = (const uint16_t*)k, a.v = (const uint16_t*)v;
    a.table = block_table, a.lens = lens, a.mask = tree_mask, a.out = out, a.lse = lse;
    a.part_ml = (float2*)w4h::ws_part(workspace);
    a.part_o = workspace ? (float*)(a.part_ml + (size_t)rows * p.S) : nullptr;
    a.q_stride = q_stride, a.page_stride = page_stride, a.token_stride = token_stride, a.head_stride = head_stride;
    a.num_pages = num_pages, a.page_shift = shift, a.table_stride = table_stride, a.max_len = max_len;
    a.scale2 = scale * kLog2e;
    a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.R = R, a.S = p.S, a.RB = p.RB;
    const bool bf16 = dtype == W4A16_BF16;
    allow_lds();
    w4h::begin_launches();
    hipLaunchKernelGGL(p.kernel[bf16], dim3((unsigned)blocks), dim3(p.threads), p.lds, (hipStream_t)stream, a);
    if (p.S > 1) {
        const dim3 grid((unsigned)((rows + 3) / 4));
        if (D == 64)
            hipLaunchKernelGGL((bf16 ? tree_merge_kernel<true, 64> : tree_merge_kernel<false, 64>), grid, dim3(256), 0, (hipStream_t)stream, a, rows);
        else if (D == 128)
            hipLaunchKernelGGL((bf16 ? tree_merge_kernel<true, 128> : tree_merge_kernel<false, 128>), grid, dim3(256), 0, (hipStream_t)stream, a, rows);
        else
            hipLaunchKernelGGL((bf16 ? tree_merge_kernel<true, 256> : tree_merge_kernel<false, 256>), grid, dim3(256), 0, (hipStream_t)stream, a, rows);
    }
    w4h::set_last_variant("tree_attn D=%d rows=%d groups=%d threads=%d blocks=%lld splits=%d row_blocks=%d lds=%zu", D,
                          p.rows, p.wk, p.threads, blocks, p.S, p.RB, p.lds);
    return w4h::launch_status();
}
