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
// Tiles of K and V go from the cache straight to LDS, whole rows of a page, NS
// tiles deep per group.  K's 16-byte chunks are permuted with the key on the
// way, so that reading one chunk of 16 keys is free of bank conflicts.
#include <math.h>

#include <atomic>
#include <type_traits>

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
constexpr size_t kMaxWorkspace = (size_t)64 << 20;

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
    float scale2;      // |scale| log2(e)
    uint32_t q_sign;   // the sign bits of two elements of q where scale is negative
    int B, T, Hq, Hkv, G, R;
    int S, RB;         // splits of the keys, blocks of rows
};

// Waits until at most N of this wave's loads are under way and its LDS reads
// are done.  The builtin and not an asm statement: the compiler then knows what
// has arrived, and does not wait for the youngest loads by itself.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}

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

// Two 16-bit values: bit 15 of each half is set where its exponent is all ones (infinity, NaN).
template <bool BF16>
__device__ __forceinline__ uint32_t overflow(uint32_t v) {
    return BF16 ? (v & 0x7f807f80u) + 0x00800080u : (v & 0x7c007c00u) + 0x04000400u;
}

template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t h) {
    constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
    return (h & kExp) == kExp;
}

// Which of a tile's 32 keys a row sees, the first of them draft d0 (negative:
// that many keys of context come first).  see: the row's mask, no bit past T.
__device__ __forceinline__ uint32_t visible(uint64_t see, int d0) {
    if (d0 >= 0) return d0 < 64 ? (uint32_t)(see >> d0) : 0u;
    return d0 <= -32 ? ~0u : (uint32_t)(see << -d0) | ((1u << -d0) - 1u);
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

// The place of a row's result.
__device__ __forceinline__ size_t out_row(const TreeArgs& a, uint32_t b, uint32_t kvh, uint32_t row) {
    const uint32_t G = a.G;
    return ((size_t)b * a.T + row / G) * a.Hq + kvh * G + row % G;
}

// Scores, maxima, sums and O are fp32.  The probabilities are rounded to the
// type of q, k and v, as the matrix unit takes them (the sum l adds them
// before that): a rounding of at most 2^-8 (bf16) or 2^-11 (f16) of each key's
// probability, averaged over the keys.  Results are off by 0.0022 of their size in
// bf16 (f16 0.00021), where rounding them alone gives 0.0017 (0.00019).
//
// One token over 150000 keys (614 MB of cache) takes 104 us, 5.9 TB/s: bound by
// memory, one workgroup of four key groups per CU (its rings take 128 of the CU's
// 160 KiB of LDS).  Four requests of 16 drafts
// over up to 4097 keys (54 MB, 80 rows a kv head) take 26 us and the merge 6:
// there a CU has one workgroup of four waves, each step (1.3 us) is a chain of
// LDS reads, scores, maxima, exponentials and the product with V that nothing
// overlaps.  Eight ring stages, eight waves in two key groups, non-temporal
// loads and other page sizes were no faster there; deeper splits pay for their parts.
template <bool BF16, int D, int RT, int WK, int WR, int NS>
__global__ __launch_bounds__(WK* WR * 64, 2) void tree_attn_kernel(TreeArgs a) {
    constexpr int DT = D / 16;                 // operand tiles of O^T
    constexpr int KS = D / 32;                 // products per score tile
    constexpr int kChunks = D / 8;             // 16-byte chunks of a key
    constexpr int kSwz = kChunks < 16 ? kChunks - 1 : 15;
    constexpr int kHalf = kTile * D * 2;       // bytes of a tile of K or of V
    constexpr int kStage = 2 * kHalf;
    constexpr int kKeys = 512 / D;             // keys per load instruction
    constexpr int kPer = kTile / kKeys / WR;   // loads of K (and of V) per wave and tile
    constexpr int kRows = 16 * RT * WR;
    // Non-temporal loads where few rows share the keys: 106 us against 117 for one token over 150000 keys, 33.5 against 36
    // for 4 drafts over 32768.  (With two blocks of rows, which read the same keys, 8 drafts over 8192 take 18.9 against 18.1.)
    // Where four waves share them, 31.7 us against 31.3 for 4 x 16 drafts over 4097: ordinary ones.
    constexpr int kAux = WR < 4 ? kAuxNT : 0;
    static_assert(kPer >= 1, "a wave loads whole instructions");
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63;
    const int kg = wave / WR, wr = wave % WR, c = lane & 15, g = lane >> 4;

    // Consecutive workgroups go to the XCDs in turn: the blocks of rows that
    // read the same keys sit 8 apart, on one XCD.
    const uint32_t u8 = blockIdx.x >> 3, row_blocks = a.RB, splits = a.S, heads = a.Hkv;
    const uint32_t rb = u8 % row_blocks, id = (u8 / row_blocks) * 8 + (blockIdx.x & 7);
    if (id >= a.B * heads * splits) return;
    const uint32_t split = id % splits, unit = id / splits, kvh = unit % heads, b = unit / heads;
    const int len = min(max(a.lens[b], 0), a.max_len), total = len + a.T;
    const int tiles = (total + kTile - 1) / kTile;
    // (tiles <= 2^25 + 2 and S <= 64: the products fit 32 bits.)
    const int t0 = (uint32_t)tiles * split / (uint32_t)a.S, t1 = (uint32_t)tiles * (split + 1) / (uint32_t)a.S;
    const int nt = t1 - t0 > kg ? (t1 - t0 - kg + WK - 1) / WK : 0;   // this group's tiles
    const int loops = (t1 - t0 + WK - 1) / WK;                        // the same for every group (barriers)

    // The page of position p, by a scalar load (the table does not change while the kernel runs).
    typedef const __attribute__((address_space(4))) int* const_ptr_t;
    const const_ptr_t table = (const_ptr_t)(a.table + (size_t)b * a.table_stride);
    auto page_of = [&](int p) {
        return min(max(table[min(p, total - 1) >> a.page_shift], 0), a.num_pages - 1);
    };
    const long long head = kvh * a.head_stride;
    uint8_t* const ring = smem + kg * NS * kStage;
    constexpr int VW = D / 32;   // dwords of a key of V per lane
    constexpr int VH = VW < 4 ? VW : 4;
    const int key_in = lane / kChunks, pos = lane % kChunks;

    // A load instruction takes whole keys of one page: its base is scalar, its
    // lane offsets constant.  (Buffer loads and not global ones: the compiler
    // waits for every global load into LDS before any LDS read.)  A wave loads
    // kSpan keys of a tile, which lie in one page, or in two halves of a page
    // each, or (short pages) are taken page by page with the other lanes off.
    constexpr int kSpan = kPer * kKeys;
    const uint32_t key_bytes = (uint32_t)(a.token_stride * 2);
    const uint32_t page_bytes = (uint32_t)((1u << a.page_shift) - 1) * key_bytes + D * 2;
    const int page_mask = (1 << a.page_shift) - 1;
    const uint32_t k_lane = 16u * (pos ^ key_in), v_lane = 16u * pos, row_lane = key_in * key_bytes;
    const bool counted = page_mask >= kKeys - 1;   // a tile then takes 2 kPer loads of a wave
    const int runs = page_mask >= kSpan - 1 ? 1 : kPer > 1 && page_mask >= kSpan / 2 - 1 ? 2 : 0;
    auto first_of = [&](int n) { return (t0 + kg + n * WK) * kTile; };   // the group's tile n
    auto load = [&](uint8_t* to, int i, const __amdgpu_buffer_rsrc_t& rk, const __amdgpu_buffer_rsrc_t& rv,
                    uint32_t row, uint32_t in_page) {
        const uint32_t k_off = k_lane ^ (16u * ((i * kKeys) & kSwz));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (lds_ptr_t)(to + i * 1024), 16, row + k_off, in_page, 0, kAux);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (lds_ptr_t)(to + kHalf + i * 1024), 16, row + v_lane, in_page, 0, kAux);
    };
    auto of_k = [&](int page) { return make_rsrc(a.k + ((long long)page * a.page_stride + head), page_bytes); };
    auto of_v = [&](int page) { return make_rsrc(a.v + ((long long)page * a.page_stride + head), page_bytes); };
    struct Pages {
        int half[2];
    };
    auto look_up = [&](int n) {   // the pages of the two halves of what this wave loads of tile n
        const int p = first_of(min(n, nt - 1)) + wr * kSpan;
        Pages pg;
        pg.half[0] = page_of(p);
        pg.half[1] = runs == 2 ? page_of(p + kSpan / 2) : pg.half[0];
        return pg;
    };
    // Tile n (past the last one, the last one again: nothing reads it) into ring slot n.
    auto issue = [&](int n, const Pages& pg) {
        uint8_t* const to = ring + (n % NS) * kStage;
        const int first = first_of(min(n, nt - 1)) + wr * kSpan;
        if (runs) {
            uint32_t in_page = (uint32_t)(first & page_mask) * key_bytes;
            __amdgpu_buffer_rsrc_t rk = of_k(pg.half[0]), rv = of_v(pg.half[0]);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (i == kPer / 2 && runs == 2) rk = of_k(pg.half[1]), rv = of_v(pg.half[1]), in_page = 0;
                load(to, wr * kPer + i, rk, rv, row_lane, in_page);
                in_page += kKeys * key_bytes;
            }
        } else {
            const int step = counted ? kKeys : page_mask + 1;
#pragma unroll 1
            for (int j = 0; j < kSpan; j += step) {
                const int page = page_of(first + j);
                const uint32_t in_page = (uint32_t)((first + j) & page_mask) * key_bytes;
                if (counted || (key_in & ~page_mask) == (j & (kKeys - 1)))
                    load(to, wr * kPer + j / kKeys, of_k(page), of_v(page), counted ? row_lane : (key_in & page_mask) * key_bytes, in_page);
            }
        }
    };

    // The rows: B operand of the scores, and each row's mask.
    const int row0 = rb * kRows + wr * RT * 16;
    u32x4_t qf[RT][KS];
    uint64_t see[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const uint32_t row = min(row0 + 16 * rt + c, a.R - 1), G = a.G;   // past the rows: the last one again, not stored
        const uint32_t tok = row / G;
        see[rt] = a.mask[(size_t)b * a.T + tok] & (~0ull >> (64 - a.T));
        const uint16_t* const qp = a.q + ((size_t)b * a.T + tok) * a.q_stride + (size_t)(kvh * G + row % G) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[rt][s] = *(const u32x4_t*)(qp + 32 * s + 8 * g);
    }
    bool any_odd = false;   // the same for the whole wave
    float4_t o[RT][DT];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -__builtin_inff(), l[rt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[rt][d] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    // One tile: scores, probabilities, product with V.  EDGE: some of its keys
    // are drafts or past the end.
    auto tile = [&](auto edge, const uint8_t* kt, const uint8_t* vt, int first) {
        constexpr bool EDGE = decltype(edge)::value;
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
        const int d0 = first - len;   // the tile's first key among the drafts (negative: context)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][rt][i & 3];
            if constexpr (EDGE) {
                const uint32_t bits = visible(see[rt], d0) >> (4 * g);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = (bits >> (16 * (i >> 2) + (i & 3))) & 1u ? x[i] : -__builtin_inff();
            }
            float top = x[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, x[i]);
            const float mn = __builtin_fmaxf(m[rt], max4(top) * a.scale2);
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
                x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], a.scale2, -base));
                sum += x[i];
            }
            l[rt] += sum;   // this lane's keys; the four lanes of a row are added at the end
#pragma unroll
            for (int j = 0; j < 4; ++j) pf[rt][j] = pack2<BF16>(x[2 * j], x[2 * j + 1]);
        }
        // V: D/16 columns of this lane's eight keys, at most eight columns at a time.
#pragma unroll
        for (int w0 = 0; w0 < VW; w0 += VH) {
            uint32_t vr[8][VH];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint8_t* const p = vt + (16 * (i >> 2) + 4 * g + (i & 3)) * D * 2 + (c * VW + w0) * 4;
                if constexpr (VH == 2) {
                    const u32x2_t v = *(const u32x2_t*)p;
                    vr[i][0] = v[0], vr[i][1] = v[1];
                } else {
                    const u32x4_t v = *(const u32x4_t*)p;
#pragma unroll
                    for (int e = 0; e < 4; ++e) vr[i][e] = v[e];
                }
            }
            if constexpr (EDGE) {
                // Keys past the end count as zeros.  A draft's infinity or NaN must
                // not reach the rows that do not see it (0 * inf): it is taken out
                // of the product, and given to the rows that do after the loop.
                uint32_t odd = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool there = d0 + 16 * (i >> 2) + 4 * g + (i & 3) < a.T;
#pragma unroll
                    for (int w = 0; w < VH; ++w) {
                        vr[i][w] = there ? vr[i][w] : 0u;
                        odd |= overflow<BF16>(vr[i][w]);
                    }
                }
                if (__builtin_amdgcn_ballot_w64((odd & 0x80008000u) != 0)) {
                    any_odd = true;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool draft = d0 + 16 * (i >> 2) + 4 * g + (i & 3) >= 0;   // context goes in as it is
#pragma unroll
                        for (int w = 0; w < VH; ++w) {
                            const uint32_t top = overflow<BF16>(vr[i][w]) & 0x80008000u;
                            vr[i][w] &= draft ? ~((top >> 15) * 0xffffu) : ~0u;
                        }
                    }
                }
            }
#pragma unroll
            for (int d = 2 * w0; d < 2 * (w0 + VH); ++d) {
                const int w = (d >> 1) - w0;
                u32x4_t va;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    va[j] = __builtin_amdgcn_perm(vr[2 * j + 1][w], vr[2 * j][w], d & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) o[rt][d] = mfma<BF16>(va, pf[rt], o[rt][d]);
            }
        }
    };

    // NS - 1 tiles are under way ahead of the one that is multiplied.  A wave
    // with a ring of its own asks for the next tile as soon as it has read the
    // last; waves that share one do so after the barrier that also says that
    // everybody's loads of this tile have arrived.
    Pages next{};   // of the tile that is issued next, asked for a step ahead
    if (nt > 0) {
        Pages pg[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) pg[n] = look_up(n);   // one latency for all
#pragma unroll
        for (int n = 0; n < NS - 1; ++n) issue(n, pg[n]);
        next = pg[NS - 1];
    }
    // The rows have arrived: only tiles' loads are waited for in the loop.
    if (counted && nt > 0) wait_loads<(NS - 1) * 2 * kPer>();
    else wait_loads<0>();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[rt][s] ^= a.q_sign;
    auto step = [&](auto edge, int n) {
        if constexpr (WR == 1) {
            wait_loads<63>();   // LDS reads only
            issue(n + NS - 1, next);
            next = look_up(n + NS);
            if (counted) wait_loads<(NS - 1) * 2 * kPer>();
            else wait_loads<0>();
        } else {
            if (counted) wait_loads<(NS - 2) * 2 * kPer>();
            else wait_loads<0>();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (n >= nt) return;   // another group has one more
            issue(n + NS - 1, next);
            next = look_up(n + NS);
        }
        if (WR > 1 && row0 >= a.R) return;   // a wave without rows only loads
        const uint8_t* const kt = ring + (n % NS) * kStage;
        tile(edge, kt, kt + kHalf, first_of(n));
    };
    // Tiles of context alone, then those with drafts or the end inside.
    const int context = min(t1, len / kTile) - t0 - kg;
    const int plain = context > 0 ? (context + WK - 1) / WK : 0;
    const int last = WR == 1 ? nt : loops;   // a barrier in each step: the same number for every group
    int n = 0;
    for (; n < plain; ++n) step(std::false_type{}, n);
    for (; n < last; ++n) step(std::true_type{}, n);
    wait_loads<0>();
    __syncthreads();
    if (any_odd) {
        // Whatever its probability, a seen infinity makes its column infinite
        // and a NaN makes it NaN: each is added as it is.
#pragma unroll 1
        for (int j = 0; j < a.T; ++j) {
            const int p = len + j, at = p / kTile - t0;
            if (at < 0 || at >= t1 - t0 || at % WK != kg) continue;   // another group's tile
            const uint16_t* const vp = a.v + (long long)page_of(p) * a.page_stride + (long long)(p & page_mask) * a.token_stride + head;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int d = 0; d < DT; d += 2) {
                    const uint32_t v = *(const uint32_t*)(vp + DT * (4 * g + q) + d);
                    const float lo = not_finite<BF16>(v) ? unpack1<BF16>(v & 0xffffu) : 0.f;
                    const float hi = not_finite<BF16>(v >> 16) ? unpack1<BF16>(v >> 16) : 0.f;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const bool sees = (see[rt] >> j) & 1;
                        o[rt][d][q] += sees ? lo : 0.f, o[rt][d + 1][q] += sees ? hi : 0.f;
                    }
                }
        }
    }

    // The groups' parts, each a sum with its own maximum: [group][row of the block].
    float* const ml = (float*)smem;                                  // [WK][kRows][2]
    float* const os = (float*)(smem + WK * kRows * 2 * sizeof(float));   // [WK][kRows][D]
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] = sum4(l[rt]);
        if (WK > 1 && g == 0) {
            float* const at = ml + (kg * kRows + wr * RT * 16 + 16 * rt + c) * 2;
            at[0] = m[rt], at[1] = l[rt];
        }
    }
    if constexpr (WK > 1) __syncthreads();
    // Where a row's sums (splits) or results go.
    auto store4 = [&](size_t at, const float4_t& v) {
        if (a.S > 1)
            *(float4_t*)(a.part_o + at) = v;
        else
            *(u32x2_t*)((uint16_t*)a.out + at) = u32x2_t{pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3])};
    };
    auto row_at = [&](uint32_t row) {
        return (a.S > 1 ? ((size_t)unit * a.R + row) * a.S + split : out_row(a, b, kvh, row)) * D;
    };
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int in_block = wr * RT * 16 + 16 * rt + c, row = rb * kRows + in_block;
        float top = m[rt], sum = WK > 1 ? 0.f : l[rt];
        if constexpr (WK > 1) {
#pragma unroll
            for (int w = 0; w < WK; ++w) top = __builtin_fmaxf(top, ml[(w * kRows + in_block) * 2]);
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                const float* const at = ml + (w * kRows + in_block) * 2;
                sum += weight_of(at[0], top) * at[1];
            }
        }
        float f = weight_of(m[rt], top);
        if (a.S == 1) f = sum == 0.f ? 0.f : f / sum;
        if (kg == 0 && g == 0 && row < a.R) {
            if (a.S > 1)
                a.part_ml[((size_t)unit * a.R + row) * a.S + split] = float2{top, sum};
            else if (a.lse)
                a.lse[out_row(a, b, kvh, row)] = sum == 0.f ? -__builtin_inff() : (top - kLift<BF16> + __builtin_log2f(sum)) * kLn2;
        }
        // Lane (c, g) holds columns DT (4g + q) + d of its row.
        float* const to = os + ((size_t)kg * kRows + in_block) * D;
        const size_t at = row_at(row);
        if (WK == 1 && row >= a.R) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int d = 0; d < DT; d += 4) {
                const float4_t v = {o[rt][d][q] * f, o[rt][d + 1][q] * f, o[rt][d + 2][q] * f, o[rt][d + 3][q] * f};
                if constexpr (WK > 1) *(float4_t*)(to + DT * (4 * g + q) + d) = v;
                else store4(at + DT * (4 * g + q) + d, v);
            }
    }
    if constexpr (WK > 1) {
        __syncthreads();
        for (int e = t * 4; e < kRows * D; e += WK * WR * 256) {
            const int row = rb * kRows + e / D;
            if (row >= a.R) break;
            float4_t v = *(const float4_t*)(os + e);
#pragma unroll
            for (int w = 1; w < WK; ++w) v += *(const float4_t*)(os + (size_t)w * kRows * D + e);
            store4(row_at(row) + e % D, v);
        }
    }
}

// Joins the S parts of each row: o = sum 2^(m_s - top) o_s / sum 2^(m_s - top) l_s.
// A workgroup per row: wave w adds parts w, w + 4, .. in that order (all loads
// of eight parts under way at once), then the four sums are added in wave
// order.  Bound by latency: a row's parts are a few KiB (2560 rows of 8 parts:
// 5.4 us; a wave per row took longer, one workgroup waited for its parts in turn).  A launch of
// its own, because the last workgroup of a unit would join 80 rows of 8 parts,
// 330 KB, on one CU: 7 us at what a CU reads.
constexpr int kMergeWaves = 4;
template <bool BF16, int D>
__global__ __launch_bounds__(kMergeWaves * 64) void tree_merge_kernel(TreeArgs a) {
    constexpr int C = D / 64;   // columns per lane
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const size_t r = blockIdx.x;
    const uint32_t R = a.R, heads = a.Hkv, unit = blockIdx.x / R, row = blockIdx.x % R;
    const float* const src = a.part_o + r * a.S * D + lane * C;
    float2 ml = float2{-__builtin_inff(), 0.f};
    if (lane < a.S) ml = a.part_ml[r * a.S + lane];
    float x[8][C];
    auto fetch = [&](int s0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int s = min(s0 + kMergeWaves * j, a.S - 1);   // past the end: a part that is not added
#pragma unroll
            for (int i = 0; i < C; ++i) x[j][i] = src[(size_t)s * D + i];
        }
    };
    fetch(wave);
    float top = ml.x;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, s));
    const float f = weight_of(ml.x, top);   // of part `lane`
    float sum = f * ml.y;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
    float v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = 0.f;
    for (int s0 = wave; s0 < a.S; s0 += 8 * kMergeWaves) {
        if (s0 != wave) fetch(s0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int s = s0 + kMergeWaves * j;
            const float w = bitcast<float>(__builtin_amdgcn_readlane(bitcast<int>(f), s & 63));
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = s < a.S ? __builtin_fmaf(w, x[j][i], v[i]) : v[i];
        }
    }
    __shared__ float parts[kMergeWaves][D];
#pragma unroll
    for (int i = 0; i < C; ++i) parts[wave][lane * C + i] = v[i];
    __syncthreads();
    const size_t at = out_row(a, unit / heads, unit % heads, row);
    const int d = threadIdx.x;
    if (d < D) {
        float o = parts[0][d];
#pragma unroll
        for (int w = 1; w < kMergeWaves; ++w) o += parts[w][d];
        o *= sum == 0.f ? 0.f : 1.0f / sum;
        ((uint16_t*)a.out)[at * D + d] = (uint16_t)pack2<BF16>(o, 0.f);
    }
    if (d == 0 && a.lse) a.lse[at] = sum == 0.f ? -__builtin_inff() : (top - kLift<BF16> + __builtin_log2f(sum)) * kLn2;
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
    long long blocks;
    size_t ws;
};

template <int D, int RT, int WK, int WR, int NS>
void use(Plan& p) {
    p.kernel[0] = tree_attn_kernel<false, D, RT, WK, WR, NS>;
    p.kernel[1] = tree_attn_kernel<true, D, RT, WK, WR, NS>;
    p.rows = 16 * RT * WR, p.wk = WK, p.threads = 64 * WK * WR;
    const size_t ring = (size_t)WK * NS * 2 * kTile * D * 2;
    const size_t join = (size_t)WK * p.rows * (2 + (WK > 1 ? D : 0)) * sizeof(float);
    p.lds = ring > join ? ring : join;
}

// The kernels of one head size: how their waves are arranged, and what a step
// (a tile for each group) of a workgroup takes in microseconds, alone on its CU and beside a
// second one, measured on MI355X with keys in HBM.
struct Shape {
    void (*use)(Plan&);
    float alone, beside;
};
template <int D>
const Shape* shapes(int& n) {
    if constexpr (D == 256) {
        static const Shape s[] = {{use<D, 1, 2, 1, 2>, 1.3f, 1.3f}, {use<D, 1, 1, 4, 4>, 1.1f, 1.1f}};
        n = 2;
        return s;
    } else {
        // D = 64 reads half the bytes a tile.
        static const Shape s[] = {{use<D, 1, 4, 1, 2>, D == 64 ? 0.6f : 1.15f, D == 64 ? 0.75f : 1.15f},
                                  {use<D, 2, 4, 1, 2>, D == 64 ? 0.75f : 1.25f, D == 64 ? 0.9f : 1.25f},
                                  {use<D, 2, 2, 2, 4>, D == 64 ? 0.8f : 1.1f, D == 64 ? 1.0f : 1.1f},
                                  {use<D, 2, 1, 4, 4>, D == 64 ? 0.7f : 0.85f, D == 64 ? 0.95f : 1.2f}};
        n = 4;
        return s;
    }
}
const Shape* shapes(int D, int& n) { return D == 64 ? shapes<64>(n) : D == 128 ? shapes<128>(n) : shapes<256>(n); }

// The kernel and the split of the keys with the least estimated time.  Few rows
// over many keys want many groups of keys, many rows a kernel whose waves share
// the keys' tiles; a split fills the GPU but pays for its parts' traffic and the merge's
// launch.  The estimate takes the longest request (max_len) for all of them.
// No kernel is left where all need more work-items than a launch takes.
Plan make_plan(int B, int T, int Hq, int Hkv, int D, int max_len) {
    constexpr double kStart = 7.0, kMerge = 5.0, kPartBytesPerUs = 4e6;   // launch to first tile and last store; merge
    const int R = T * (Hq / Hkv), cus = w4h::cu_count();
    const long long units = (long long)B * Hkv, tiles = ((long long)max_len + T + kTile - 1) / kTile;
    Plan best{};
    double least = 0;
    int n;
    const Shape* const sh = shapes(D, n);
    for (int i = 0; i < n; ++i) {
        Plan p{};
        sh[i].use(p);
        p.units = units;
        p.RB = (R + p.rows - 1) / p.rows;
        const int occupancy = p.lds * 2 <= (size_t)kMaxDynamicLds ? 2 : 1;
        // Splits worth a look: none, few, and those that fill every CU once or to its occupancy, or halfway.
        const long long full = cus / (units * p.RB), most = (long long)cus * occupancy / (units * p.RB);
        for (long long S : {1LL, 2LL, 3LL, full / 2, full, most}) {
            S = S < kMaxSplit ? S : kMaxSplit;
            S = S < tiles / (2 * p.wk) ? S : tiles / (2 * p.wk);   // two tiles at least for each group
            S = S < 1 ? 1 : S;
            p.ws = S > 1 ? w4h::ws_bytes((size_t)units * R * S * (D + 2) * sizeof(float)) : 0;
            p.blocks = (units * S + 7) / 8 * 8 * p.RB;
            if (p.ws > kMaxWorkspace || p.blocks * p.threads > kMaxLanes || (S > 1 && units * R * kMergeWaves * 64 > kMaxLanes)) continue;
            const double wgs = (double)units * p.RB * S, steps = ceil((double)tiles / S / p.wk);
            const double rounds = ceil(wgs / ((double)cus * occupancy));
            double t = rounds * (kStart + steps * (wgs > cus ? sh[i].beside : sh[i].alone));
            if (S > 1) t += kMerge + (double)units * R * S * D * 8 / kPartBytesPerUs;
            if (best.rows == 0 || t < least) {
                least = t;
                best = p;
                best.S = (int)S;
            }
        }
    }
    return best;
}

// The kernels' dynamic LDS may pass the default limit: said once per process and device.
void allow_lds() {
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices || done[dev].load(std::memory_order_acquire)) return;
    for (int D : {64, 128, 256}) {
        int n;
        const Shape* const sh = shapes(D, n);
        for (int i = 0; i < n; ++i) {
            Plan p{};
            sh[i].use(p);
            for (kernel_t k : p.kernel)
                (void)hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicLds);
        }
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
    const Plan p = make_plan(B, T, Hq, Hkv, D, max_len);
    if (!p.rows) return W4A16_ERR_UNSUPPORTED;
    *bytes = p.ws;
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
        (unsigned long long)page_size * (unsigned long long)token_stride >= (1ull << 30) || page_stride % 8 ||
        token_stride % 8 || head_stride % 8 || !(scale == scale) || scale - scale != 0.f)
        return W4A16_ERR_SHAPE;
    if (!w4h::aligned16(q) || !w4h::aligned16(k) || !w4h::aligned16(v) || !w4h::aligned16(out) ||
        !w4h::aligned16(workspace) || ((uintptr_t)lens & 3) || ((uintptr_t)block_table & 3) ||
        ((uintptr_t)tree_mask & 7) || ((uintptr_t)lse & 3))
        return W4A16_ERR_ALIGN;
    const Plan p = make_plan(B, T, Hq, Hkv, D, max_len);
    if (!p.rows) return W4A16_ERR_UNSUPPORTED;
    const int R = T * (Hq / Hkv);
    const long long rows = p.units * R;
    if (p.ws && !workspace) return W4A16_ERR_NULL;
    if (workspace_bytes < p.ws) return W4A16_ERR_WORKSPACE;
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    TreeArgs a{};
    a.q = (const uint16_t*)q, a.k = (const uint16_t*)k, a.v = (const uint16_t*)v;
    a.table = block_table, a.lens = lens, a.mask = tree_mask, a.out = out, a.lse = lse;
    // The sums first: a multiple of 64 floats, so they and the pairs behind them are aligned for any number of rows and splits.
    a.part_o = (float*)w4h::ws_part(workspace);
    a.part_ml = workspace ? (float2*)(a.part_o + (size_t)rows * p.S * D) : nullptr;
    a.q_stride = q_stride, a.page_stride = page_stride, a.token_stride = token_stride, a.head_stride = head_stride;
    a.num_pages = num_pages, a.page_shift = shift, a.table_stride = table_stride, a.max_len = max_len;
    a.scale2 = fmaxf(fabsf(scale) * kLog2e, 0x1p-126f);   // not 0: -inf marks what a row does not see
    a.q_sign = scale < 0.f ? 0x80008000u : 0u;
    a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.R = R, a.S = p.S, a.RB = p.RB;
    const bool bf16 = dtype == W4A16_BF16;
    allow_lds();
    w4h::begin_launches();
    hipLaunchKernelGGL(p.kernel[bf16], dim3((unsigned)p.blocks), dim3(p.threads), p.lds, (hipStream_t)stream, a);
    if (p.S > 1) {
        const kernel_t merge = D == 64    ? (bf16 ? tree_merge_kernel<true, 64> : tree_merge_kernel<false, 64>)
                               : D == 128 ? (bf16 ? tree_merge_kernel<true, 128> : tree_merge_kernel<false, 128>)
                                          : (bf16 ? tree_merge_kernel<true, 256> : tree_merge_kernel<false, 256>);
        hipLaunchKernelGGL(merge, dim3((unsigned)rows), dim3(kMergeWaves * 64), 0, (hipStream_t)stream, a);
    }
    w4h::note_variant("%s D=%lld rows=%lld groups=%lld threads=%lld blocks=%lld splits=%lld row_blocks=%lld lds=%lld",
                      "tree_attn", D, p.rows, p.wk, p.threads, p.blocks, p.S, p.RB, p.lds);
    return w4h::launch_status();
}
