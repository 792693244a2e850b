// prefix_attn.hip -- attention of a batch that shares a long prefix, over a
// paged cache.
//
// One launch takes two kinds of work side by side, and a second one joins their
// parts.  Prefix work is bound by the matrix units: the rows of all requests
// (B T G of a kv head) against the same keys, in blocks of 128 rows whose four
// waves share tiles of 32 keys in LDS.  Own work is bound by memory: the T G
// rows of one request against its own keys, whose waves take tiles in turn and
// load them straight into registers.  Where the prefix is short the own work
// takes it too (each request reads it again, from the caches), which saves the parts.
//
// Products.  Scores are computed transposed, S^T = K Q^T, so that a lane holds one
// row's scores, in the layout in which O^T = V^T P^T takes P as its B operand
// once the slots of k are named after the keys that the lane holds.  V^T comes from
// LDS by transposing reads (prefix work), or (own work) lane r of operand tile t takes column
// (D/16) r + t, so that it loads consecutive columns of each key and pairs keys up with byte permutes.
//
// Measured (a call among others, three sets of inputs in turn, from a graph or not): 256 requests of 4 drafts, 40 query heads
// of 128, over 16384 shared keys in 406 to 415 us: 840 to 858 TFLOP/s, of 1214 that a large library product reaches; the
// softmax between the products takes the rest.  8 requests behind a document of 131000 keys (8 key/value heads), 1000 of
// their own, in 96.5 us: 5.8 TB/s, the cache read once.
#include "attn_common.h"
#include "../../include/prefix_attn.h"

using namespace w4k;

namespace {

constexpr int kTile = 32;              // keys per tile
constexpr int kWaves = 4;
constexpr int kBlockRows = 32 * kWaves;   // rows of a workgroup of prefix work
constexpr int kStages = 4;             // ring stages of prefix work
constexpr int kMaxParts = 256;
constexpr size_t kMaxPartBytes = (size_t)128 << 20;

struct PrefixArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int* prefix_table;
    const int* prefix_len;
    const int* table;
    const int* lens;
    const uint64_t* mask;
    uint16_t* out;
    float* lse;
    float* part_o;     // [row of out][part][D] sums that are not divided yet
    float2* part_ml;   // [row of out][part] maximum (log2 units) and sum
    long long q_stride, page_stride, token_stride, head_stride;
    int num_pages, page_shift, table_stride;
    int max_prefix, max_len;
    float scale2;      // |scale| log2(e)
    uint32_t q_sign;   // the sign bits of two elements of q where scale is negative
    int B, T, Hq, Hkv, G;
    int SP, RB;        // prefix work: splits of the keys, blocks of rows; SP = 0: the own work takes the prefix
    int SO, RO;        // own work: splits, blocks of rows
    int parts;         // SP + SO
    uint32_t prefix_groups, own_groups;   // groups of eight workgroups
    int own_first;     // the own work's workgroups take longer
};

// Probabilities are 2^(x - m + kLift): in f16 that keeps them normal down to
// 2^-26 of the largest, where a long context's many small ones would otherwise fall
// on the subnormal grid.  A row's maximum m is raised only once a score passes it by
// kSlack, so that O is seldom rescaled: probabilities stay below 2^(kLift + kSlack), in
// f16's range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 12.f;
template <bool BF16>
constexpr float kSlack = BF16 ? 8.f : 3.f;

// A score's product with scale2 enters the exponent unrounded, the maximum rounded: past kFar (log2 units) that
// difference could pass f16's range (and from 2^31 on bf16's).  There every tile rounds each product like the
// maximum first, so that the largest one's exponent is kLift again.
constexpr float kFar = 0x1p20f;
__device__ __forceinline__ bool is_far(float m) { return __builtin_fabsf(m) > kFar && m != -__builtin_inff(); }
// What a score has to pass for the maximum m to be raised.
template <bool BF16>
__device__ __forceinline__ float limit_of(float m) {
    return __builtin_fabsf(m) > kFar ? -__builtin_inff() : m + kSlack<BF16>;
}
template <bool BF16>
__device__ __forceinline__ float far_exponent(float x, float scale2, float m) {
#pragma clang fp contract(off)
    const float y = x * scale2;
    return y - (m == -__builtin_inff() ? 0.f : m) + kLift<BF16>;
}

typedef float float16_t __attribute__((ext_vector_type(16)));
typedef short v4i16_t __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ float16_t mfma32(const u32x4_t& a, const u32x4_t& b, const float16_t& c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(bitcast<bf16x8_t>(a), bitcast<bf16x8_t>(b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(bitcast<half8_t>(a), bitcast<half8_t>(b), c, 0, 0, 0);
}

// The other half-wave's x beside this one's.
__device__ __forceinline__ float max2(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(bitcast<uint32_t>(x), bitcast<uint32_t>(x), false, false);
    return __builtin_fmaxf(bitcast<float>((uint32_t)a[0]), bitcast<float>((uint32_t)a[1]));
}
__device__ __forceinline__ float sum2(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(bitcast<uint32_t>(x), bitcast<uint32_t>(x), false, false);
    return bitcast<float>((uint32_t)a[0]) + bitcast<float>((uint32_t)a[1]);
}

typedef const __attribute__((address_space(4))) int* const_ptr_t;

// The page of position p of a table whose last position is end - 1, by a scalar
// load (the tables do not change while the kernel runs).
__device__ __forceinline__ int page_of(const PrefixArgs& a, const int* table, int p, int end) {
    return min(max(((const_ptr_t)table)[min(p, end - 1) >> a.page_shift], 0), a.num_pages - 1);
}

// V's 64-byte pieces of a key change places with the key, so that the four keys that a
// transposing read takes together lie on different banks.
template <int D>
__device__ __forceinline__ uint32_t v_swizzle(uint32_t key) {
    return D == 64 ? (key >> 1) & 1 : key & 3;
}

// The first of n tiles that part i of s takes (the first n % s parts take one more).
__device__ __forceinline__ int share(int n, int s, int i) {
    const int each = (uint32_t)n / (uint32_t)s;
    return i * each + min(i, n - s * each);
}

// An infinity among the values that a row sees makes its column infinite however small its
// probability, but the products (and the weights of parts and waves) make NaN of an infinity times 0.  So columns
// d .. d + N - 1 of a row that came out as NaN, its probabilities being numbers, are settled by the values
// themselves: NaN where there is a NaN or both infinities, else the infinity.  Seldom, and slow: up to all keys are read
// again (a NaN at the prefix's end that 40960 rows of 16384 keys see: 59 ms; one that 448 x 8 rows of 4099 see: 1.9).
template <bool BF16, int N>
__device__ __forceinline__ void settle(const PrefixArgs& a, size_t tok, uint32_t kvh, int d, float* v) {
    const uint32_t b = tok / (uint32_t)a.T;
    const int P = min(max(a.prefix_len[0], 0), a.max_prefix), len = min(max(a.lens[b], 0), a.max_len), page_mask = (1 << a.page_shift) - 1;
    const uint64_t see = a.mask[tok] & (~0ull >> (64 - a.T));
    uint32_t seen[N];   // bit 0: +infinity, 1: -infinity, 2: NaN
#pragma unroll
    for (int i = 0; i < N; ++i) seen[i] = 0;
#pragma unroll 1
    for (int own = 1; own >= 0; --own) {   // the shorter first: a NaN ends it
        const int n = own ? len + a.T : P;
        const int* const table = own ? a.table + (size_t)b * a.table_stride : a.prefix_table;
#pragma unroll 1
        for (int p0 = 0; p0 < n; p0 += 8) {
            uint16_t x[8][N];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int p = min(p0 + j, n - 1), page = min(max(table[p >> a.page_shift], 0), a.num_pages - 1);
                const uint16_t* const at = a.v + (long long)page * a.page_stride + (long long)(p & page_mask) * a.token_stride + kvh * a.head_stride + d;
                __builtin_memcpy(x[j], __builtin_assume_aligned(at, 2 * N), 2 * N);
            }
            bool open = false;
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int p = min(p0 + j, n - 1);
                    const float y = unpack1<BF16>(x[j][i]);
                    const bool sees = !own || p < len || ((see >> (p - len)) & 1);
                    if (sees && not_finite<BF16>(x[j][i])) seen[i] |= y != y ? 4u : y > 0.f ? 1u : 2u;
                }
                open |= v[i] != v[i] && seen[i] < 3u;
            }
            if (!__builtin_amdgcn_ballot_w64(open)) return;   // NaN, all that are left
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (v[i] != v[i] && (seen[i] == 1u || seen[i] == 2u)) v[i] = seen[i] == 1u ? __builtin_inff() : -__builtin_inff();
}

// ------------------------------------------------------------- prefix work

// Workgroup (unit, rb): keys [tile t0, tile t1) of the prefix for kv head unit / SP, rows rb * 128 .. of the B T G.
template <bool BF16, int D>
__device__ __forceinline__ void prefix_work(const PrefixArgs& a, uint32_t unit, uint32_t rb, uint8_t* smem) {
    constexpr int NS = kStages;
    constexpr int NT = D / 32;                 // operand tiles of O^T
    constexpr int KS = D / 16;                 // products per score tile
    constexpr int kChunks = D / 8;             // 16-byte chunks of a key
    constexpr int kSwz = kChunks < 16 ? kChunks - 1 : 15;
    constexpr int kHalf = kTile * D * 2;       // bytes of a tile of K or of V
    constexpr int kStage = 2 * kHalf;
    constexpr int kKeys = 512 / D;             // keys per load instruction
    constexpr int kSpan = kTile / kWaves;      // keys that a wave loads of a tile: in one page
    constexpr int kPer = kSpan / kKeys;        // its loads of K (and of V)
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63, c = lane & 31, hi = lane >> 5;
    const uint32_t split = unit % (uint32_t)a.SP, kvh = unit / (uint32_t)a.SP;
    const int P = min(max(a.prefix_len[0], 0), a.max_prefix), tiles = (P + kTile - 1) / kTile;
    const int t0 = share(tiles, a.SP, split), t1 = share(tiles, a.SP, split + 1);
    const long long head = kvh * a.head_stride;
    const uint32_t key_bytes = (uint32_t)(a.token_stride * 2);
    const int page_mask = (1 << a.page_shift) - 1;
    const uint32_t page_bytes = (uint32_t)page_mask * key_bytes + D * 2;
    const int key_in = lane / kChunks, pos = lane % kChunks;
    const bool once = a.RB == 1;   // nobody else reads these keys

    const uint32_t rows = (uint32_t)a.B * a.T * a.G, row0 = rb * kBlockRows + wave * 32, G = a.G;
    const uint32_t row = min(row0 + c, rows - 1);      // past the rows: the last one again, not stored
    const size_t tok = row / G, out_row = tok * a.Hq + kvh * G + row % G;
    u32x4_t qf[KS];
    {
        const uint16_t* const qp = a.q + tok * a.q_stride + (size_t)(kvh * G + row % G) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = *(const u32x4_t*)(qp + 16 * s + 8 * hi);
    }
    auto look_up = [&](int n) { return page_of(a, a.prefix_table, min(n, t1 - 1) * kTile + wave * kSpan, P); };
    // Tile n (past the last one, the last one again: nothing reads it) into its ring slot.
    auto issue = [&](int n, int page) {
        uint8_t* const to = smem + (n - t0) % NS * kStage + wave * kPer * 1024;
        const int first = min(n, t1 - 1) * kTile + wave * kSpan;
        const uint32_t in_page = (uint32_t)(first & page_mask) * key_bytes;
        const long long at = (long long)page * a.page_stride + head;
        const __amdgpu_buffer_rsrc_t rk = make_rsrc(a.k + at, page_bytes), rv = make_rsrc(a.v + at, page_bytes);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t key = key_in + i * kKeys, k_off = 16u * (pos ^ ((wave * kSpan + key) & kSwz)), v_off = 16u * (pos ^ (4 * v_swizzle<D>(key)));
            if (once) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (lds_ptr_t)(to + i * 1024), 16, key * key_bytes + k_off, in_page, 0, kAuxNT);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (lds_ptr_t)(to + kHalf + i * 1024), 16, key * key_bytes + v_off, in_page, 0, kAuxNT);
            } else {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (lds_ptr_t)(to + i * 1024), 16, key * key_bytes + k_off, in_page, 0, 0);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (lds_ptr_t)(to + kHalf + i * 1024), 16, key * key_bytes + v_off, in_page, 0, 0);
            }
        }
    };
    float16_t o[NT];
    float m = -__builtin_inff(), l = 0.f, limit = m, base = 0.f;   // base: of the exponents, m - kLift
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    int next = 0;
    if (t0 < t1) {
        int page[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) page[n] = look_up(t0 + n);
#pragma unroll
        for (int n = 0; n < NS - 1; ++n) issue(t0 + n, page[n]);
        next = page[NS - 1];
        wait_loads<(NS - 1) * 2 * kPer>();   // the rows have arrived
    } else {
        wait_loads<0>();
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) qf[s] ^= a.q_sign;

    // K of a tile: the scores' A operand.  Heads of 256 leave no registers for reading it (and
    // all of V) ahead: they read pieces when they are needed.
    constexpr bool kAhead = D < 256;
    constexpr int KP = kAhead ? KS : 8;
    u32x4_t kf[KP];
    auto read_k = [&](const uint8_t* kt, int s0) {
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const int s = s0 + i;
            kf[i] = *(const u32x4_t*)(kt + c * D * 2 + 16 * ((2 * s + hi) ^ (c & kSwz)));
        }
    };
    // V^T of a tile: lane (c, hi) of operand tile d and half h has column 32 d + c of keys 16 h + 8 j + 4 hi + i
    // (word 2 j + i / 2).  A transposing read of 16 lanes takes 16 columns of four keys: lane l asks
    // for columns 4 (l % 4) .. of key l / 4 and gets column l of the four.
    u32x4_t va[kAhead ? 2 : 1][NT];
    const uint32_t v_key = 4 * hi + ((lane & 15) >> 2), v_lane = v_key * D * 2 + 64 * v_swizzle<D>(v_key) + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
    auto read_v = [&](const uint8_t* vt, int h) {
        typedef __attribute__((address_space(3))) v4i16_t* tr_ptr_t;
#pragma unroll
        for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u32x2_t v = bitcast<u32x2_t>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr_t)(vt + (v_lane ^ (64 * d)) + (16 * h + 8 * j) * D * 2)));
                va[kAhead ? h : 0][d][2 * j] = v[0], va[kAhead ? h : 0][d][2 * j + 1] = v[1];
            }
    };
    // One tile, whose K is in registers: scores, probabilities, product with V.  Score i of lane
    // (c, hi) is that of key 8 (i / 4) + 4 hi + i % 4.  V is read beside the softmax, the next
    // tile's K (after the barrier that says it has arrived) beside the product with V.
    // Products go before the other wave's softmax (priorities: 414 -> 404 us for 1024 x 40 rows over 16384 keys).
    // EDGE: some of its keys are past the end (a copy of its own: behind branches, whole tiles take 4 % longer).
    auto tile = [&](auto is_edge, const uint8_t* kt, const uint8_t* vt, int first, auto turn) {
        constexpr bool EDGE = decltype(is_edge)::value;
        float16_t x;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (!kAhead && s % KP == 0) read_k(kt, s);
            x = mfma32<BF16>(kf[s % KP], qf[s], x);
        }
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        read_v(vt, 0);
        if constexpr (kAhead) read_v(vt, 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (EDGE) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = first + 8 * (i >> 2) + 4 * hi + (i & 3) < P ? x[i] : -__builtin_inff();
        }
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, x[i]);
        const float mn = max2(top) * a.scale2;
        float factor = a.scale2, less = base;
        if (__builtin_amdgcn_ballot_w64(mn > limit)) {
            const float up = __builtin_fmaxf(m, mn), f = weight_of(m, up);
            l *= f;
#pragma unroll
            for (int d = 0; d < NT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= f;
            m = up, limit = limit_of<BF16>(m);
            less = base = m == -__builtin_inff() ? 0.f : m - kLift<BF16>;
            if (__builtin_amdgcn_ballot_w64(is_far(m))) {
                factor = 1.f, less = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = far_exponent<BF16>(x[i], a.scale2, m);
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], factor, -less));
            sum += x[i];
        }
        l += sum;   // this lane's keys; the two lanes of a row are added at the end
        u32x4_t pf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) pf[h][j] = pack2<BF16>(x[8 * h + 2 * j], x[8 * h + 2 * j + 1]);
        __builtin_amdgcn_s_setprio(1);
        auto multiply = [&](int h) {
            if constexpr (EDGE) {   // 0 times what lies past the end could be NaN
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int left = P - first - (16 * h + 8 * (w >> 1) + 4 * hi + 2 * (w & 1));   // keys of the word that are there
                    const uint32_t keep = left >= 2 ? ~0u : left == 1 ? 0xffffu : 0u;
#pragma unroll
                    for (int d = 0; d < NT; ++d) va[kAhead ? h : 0][d][w] &= keep;
                }
            }
#pragma unroll
            for (int d = 0; d < NT; ++d) o[d] = mfma32<BF16>(va[kAhead ? h : 0][d], pf[h], o[d]);
            __builtin_amdgcn_sched_barrier(0);
        };
        if constexpr (!kAhead) {
            multiply(0);
            read_v(vt, 1);
        }
        wait_loads<63>();   // V has arrived: its place in the ring may be loaded anew after the barrier
        turn();
        if constexpr (kAhead) multiply(0);
        multiply(1);
    };
    auto slot = [&](int n) { return smem + (n - t0) % NS * kStage; };
    // Tile n + 1 has arrived for everybody, and nobody needs tile n - 1's place any more.
    auto arrive = [&](int n) {
        wait_loads<(NS - 3) * 2 * kPer>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(n + NS - 1, next);
        next = look_up(n + NS);
    };
    const bool idle = row0 >= rows;   // a wave without rows only loads
    if (t0 < t1) {
        wait_loads<(NS - 2) * 2 * kPer>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kAhead && !idle) read_k(slot(t0), 0);
    }
    auto step = [&](auto is_edge, int n) {
        if (idle) {
            arrive(n);
            return;
        }
        tile(is_edge, slot(n), slot(n) + kHalf, n * kTile, [&] {
            arrive(n);
            if constexpr (kAhead) read_k(slot(n + 1), 0);   // past the last tile: the last one again
        });
    };
    int n = t0;
    for (const int plain = min(t1, P / kTile); n < plain; ++n) step(std::false_type{}, n);
    for (; n < t1; ++n) step(std::true_type{}, n);
    wait_loads<0>();   // nothing may land in LDS after the workgroup's end
    if (row0 + c >= rows) return;
    l = sum2(l);
    const size_t part = out_row * a.parts + split;
    if (hi == 0) a.part_ml[part] = float2{m, l};
    // o[d][i] is column 32 d + 8 (i / 4) + 4 hi + i % 4.
    float* const to = a.part_o + part * D + 4 * hi;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) *(float4_t*)(to + 32 * d + 2 * i) = float4_t{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
}

// ---------------------------------------------------------------- own work

// Workgroup (id, rb): request, kv head and split id; rows rb * 16 RT .. of the request's T G.  Tiles are the
// prefix's (where SP = 0) and the request's own; wave w takes tiles t0 + w, t0 + w + 4, ..
template <bool BF16, int D, int RT>
__device__ __forceinline__ void own_work(const PrefixArgs& a, uint32_t id, uint32_t rb, uint8_t* smem) {
    constexpr int DT = D / 16, KS = D / 32;
    constexpr int VW = D / 32;            // dwords of a key of V per lane
    constexpr int kRows = 16 * RT;
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63, c = lane & 15, g = lane >> 4;
    const uint32_t split = id % (uint32_t)a.SO, unit = id / (uint32_t)a.SO, kvh = unit % (uint32_t)a.Hkv, b = unit / (uint32_t)a.Hkv;
    const int len = min(max(a.lens[b], 0), a.max_len), own_tiles = (len + a.T + kTile - 1) / kTile;
    const int P = a.SP ? 0 : min(max(a.prefix_len[0], 0), a.max_prefix), prefix_tiles = (P + kTile - 1) / kTile;
    const int tiles = prefix_tiles + own_tiles;
    const int t0 = share(tiles, a.SO, split), t1 = share(tiles, a.SO, split + 1);
    const int* const own_table = a.table + (size_t)b * a.table_stride;
    const long long head = kvh * a.head_stride;
    const uint32_t key_bytes = (uint32_t)(a.token_stride * 2);
    const int page_mask = (1 << a.page_shift) - 1;
    const uint32_t page_bytes = (uint32_t)page_mask * key_bytes + D * 2;

    // The rows: B operand of the scores, and each row's mask.
    const uint32_t R = (uint32_t)a.T * a.G, G = a.G, row0 = rb * kRows;
    u32x4_t qf[RT][KS];
    uint64_t see[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const uint32_t row = min(row0 + 16 * rt + c, R - 1);   // past the rows: the last one again, not stored
        const size_t tok = (size_t)b * a.T + row / G;
        see[rt] = a.mask[tok] & (~0ull >> (64 - a.T));
        const uint16_t* const qp = a.q + tok * a.q_stride + (size_t)(kvh * G + row % G) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[rt][s] = *(const u32x4_t*)(qp + 32 * s + 8 * g) ^ a.q_sign;
    }
    float4_t o[RT][DT];
    float m[RT], l[RT], limit[RT], base[RT];   // base: of the exponents, m - kLift
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = limit[rt] = -__builtin_inff(), l[rt] = base[rt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[rt][d] = float4_t{0.f, 0.f, 0.f, 0.f};
    }
    bool any_odd = false;   // the same for the whole wave

    // A tile's place: halves of 16 keys lie in one page each (pages have 16 or more).
    struct Place {
        int first, len, T;      // its first position, context and drafts of its segment
        long long at[2];        // elements from the cache's start to the halves' pages
        uint32_t in_page[2];    // bytes
    };
    auto place = [&](int i) {
        Place p;
        const bool shared = i < prefix_tiles;
        p.first = (shared ? i : i - prefix_tiles) * kTile;
        p.len = shared ? P : len, p.T = shared ? 0 : a.T;
        const int* const table = shared ? a.prefix_table : own_table;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = p.first + 16 * h;
            p.at[h] = (long long)page_of(a, table, at, p.len + p.T) * a.page_stride + head;
            p.in_page[h] = (uint32_t)(at & page_mask) * key_bytes;
        }
        return p;
    };
    u32x4_t kf[2][KS];
    uint32_t vr[8][VW];
    auto load_k = [&](const Place& p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __amdgpu_buffer_rsrc_t r = make_rsrc(a.k + p.at[h], page_bytes);
#pragma unroll
            for (int s = 0; s < KS; ++s)
                kf[h][s] = bitcast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(r, c * key_bytes + 16 * g + 64 * s, p.in_page[h], 0));
        }
    };
    auto load_v = [&](const Place& p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int h = i >> 2;
            const __amdgpu_buffer_rsrc_t r = make_rsrc(a.v + p.at[h], page_bytes);
            const uint32_t off = (4 * g + (i & 3)) * key_bytes + c * VW * 4;
            if constexpr (VW == 2) {
                const u32x2_t v = bitcast<u32x2_t>(__builtin_amdgcn_raw_buffer_load_b64(r, off, p.in_page[h], 0));
                vr[i][0] = v[0], vr[i][1] = v[1];
            } else {
#pragma unroll
                for (int w = 0; w < VW; w += 4) {
                    const u32x4_t v = bitcast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(r, off + 4 * w, p.in_page[h], 0));
#pragma unroll
                    for (int e = 0; e < 4; ++e) vr[i][w + e] = v[e];
                }
            }
        }
    };
    // One tile; its keys are in registers, its values and the next tile's keys on their way.
    // What drafts and the end need stands behind branches: a second copy of this code would have to
    // be fetched, which a short call waits for (8 requests of 7 drafts, heads of 256: 10.0 -> 7.1 us).
    auto tile = [&](const Place& p, const Place& next, bool more) {
        const bool edge = p.first + kTile > p.len;   // some of its keys are drafts or past the end
        float4_t sc[2][RT];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                sc[h][rt] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < KS; ++s) sc[h][rt] = mfma<BF16>(kf[h][s], qf[rt][s], sc[h][rt]);
            }
        if (more) load_k(next);
        u32x4_t pf[RT];
        const int d0 = p.first - p.len;   // the tile's first key among the drafts (negative: context)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][rt][i & 3];
            if (edge) {
                const uint32_t bits = visible(p.T ? see[rt] : 0, d0) >> (4 * g);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = (bits >> (16 * (i >> 2) + (i & 3))) & 1u ? x[i] : -__builtin_inff();
            }
            float top = x[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, x[i]);
            const float mn = max4(top) * a.scale2;
            float factor = a.scale2, less = base[rt];
            if (__builtin_amdgcn_ballot_w64(mn > limit[rt])) {
                const float up = __builtin_fmaxf(m[rt], mn), f = weight_of(m[rt], up);
                l[rt] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[rt][d][q] *= f;
                m[rt] = up, limit[rt] = limit_of<BF16>(up);
                less = base[rt] = up == -__builtin_inff() ? 0.f : up - kLift<BF16>;
                if (__builtin_amdgcn_ballot_w64(is_far(up))) {
                    factor = 1.f, less = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = far_exponent<BF16>(x[i], a.scale2, up);
                }
            }
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], factor, -less));
                sum += x[i];
            }
            l[rt] += sum;
#pragma unroll
            for (int j = 0; j < 4; ++j) pf[rt][j] = pack2<BF16>(x[2 * j], x[2 * j + 1]);
        }
        if (edge) {
            // Keys past the end count as zeros.  A draft's infinity or NaN must not
            // reach the rows that do not see it (0 * inf): it is taken out of the
            // product, and given to the rows that do after the loop.
            uint32_t odd = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool there = d0 + 16 * (i >> 2) + 4 * g + (i & 3) < p.T;
#pragma unroll
                for (int w = 0; w < VW; ++w) {
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
                    for (int w = 0; w < VW; ++w) {
                        const uint32_t bad = overflow<BF16>(vr[i][w]) & 0x80008000u;
                        vr[i][w] &= draft ? ~((bad >> 15) * 0xffffu) : ~0u;
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
        if (more) load_v(next);
    };
    int i = t0 + wave;
    if (i < t1) {
        Place p = place(i);
        load_k(p);
        load_v(p);
#pragma unroll 1
        for (; i < t1; i += kWaves) {
            const bool more = i + kWaves < t1;
            const Place next = more ? place(i + kWaves) : p;
            tile(p, next, more);
            p = next;
        }
    }
    if (any_odd) {
        // Whatever its probability, a seen infinity makes its column infinite
        // and a NaN makes it NaN: each is added as it is.
#pragma unroll 1
        for (int j = 0; j < a.T; ++j) {
            const int p = len + j, at = prefix_tiles + p / kTile - t0;
            if (at < 0 || at >= t1 - t0 || at % kWaves != wave) continue;   // another wave's tile
            const uint16_t* const vp = a.v + (long long)page_of(a, own_table, p, len + a.T) * a.page_stride + (long long)(p & page_mask) * a.token_stride + head;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int d = 0; d < DT; d += 2) {
                    const uint32_t v = *(const uint32_t*)(vp + DT * (4 * g + q) + d);
                    const float lo = not_finite<BF16>(v) ? unpack1<BF16>(v & 0xffffu) : 0.f;
                    const float up = not_finite<BF16>(v >> 16) ? unpack1<BF16>(v >> 16) : 0.f;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const bool sees = (see[rt] >> j) & 1;
                        o[rt][d][q] += sees ? lo : 0.f, o[rt][d + 1][q] += sees ? up : 0.f;
                    }
                }
        }
    }
    // The waves' parts, each a sum with its own maximum, joined in wave order.
    float* const ml = (float*)smem;                                          // [waves][kRows][2]
    constexpr int kPitch = D + 4;                                            // rows side by side in the lanes: not on the same banks
    float* const os = (float*)(smem + kWaves * kRows * 2 * sizeof(float));   // [waves][kRows][kPitch]
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] = sum4(l[rt]);
        if (g == 0) {
            float* const at = ml + (wave * kRows + 16 * rt + c) * 2;
            at[0] = m[rt], at[1] = l[rt];
        }
    }
    __syncthreads();
    const bool direct = a.parts == 1;
    auto out_row = [&](uint32_t row) { return ((size_t)b * a.T + row / G) * a.Hq + kvh * G + row % G; };
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const uint32_t in_block = 16 * rt + c, row = row0 + in_block;
        float top = m[rt], sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = __builtin_fmaxf(top, ml[(w * kRows + in_block) * 2]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float* const at = ml + (w * kRows + in_block) * 2;
            sum += weight_of(at[0], top) * at[1];
        }
        float f = weight_of(m[rt], top);
        if (direct) f = sum == 0.f ? 0.f : f / sum;
        if (wave == 0 && g == 0 && row < R) {
            if (!direct) a.part_ml[out_row(row) * a.parts + a.SP + split] = float2{top, sum};
            else if (a.lse) a.lse[out_row(row)] = sum == 0.f ? -__builtin_inff() : (top - kLift<BF16> + __builtin_log2f(sum)) * kLn2;
        }
        // Lane (c, g) holds columns DT (4 g + q) + d of its row.
        float* const to = os + ((size_t)wave * kRows + in_block) * kPitch;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int d = 0; d < DT; d += 4)
                *(float4_t*)(to + DT * (4 * g + q) + d) = float4_t{o[rt][d][q] * f, o[rt][d + 1][q] * f, o[rt][d + 2][q] * f, o[rt][d + 3][q] * f};
    }
    __syncthreads();
    for (int e = t * 4; e < kRows * D; e += kWaves * 256) {
        const uint32_t row = row0 + e / D;
        if (row >= R) break;
        const float* const from = os + (e / D) * kPitch + e % D;
        float4_t v = *(const float4_t*)from;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += *(const float4_t*)(from + (size_t)w * kRows * kPitch);
        if (direct && (v[0] != v[0] || v[1] != v[1] || v[2] != v[2] || v[3] != v[3])) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) sum += ml[(w * kRows + e / D) * 2 + 1];
            float y[4] = {v[0], v[1], v[2], v[3]};
            if (sum - sum == 0.f) settle<BF16, 4>(a, (size_t)b * a.T + row / G, kvh, e % D, y);
            v = float4_t{y[0], y[1], y[2], y[3]};
        }
        if (direct)
            *(u32x2_t*)(a.out + out_row(row) * D + e % D) = u32x2_t{pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3])};
        else
            *(float4_t*)(a.part_o + (out_row(row) * a.parts + a.SP + split) * D + e % D) = v;
    }
}

// Scores, maxima, sums and O are fp32.  The probabilities are rounded to the
// type of q, k and v, as the matrix unit takes them (the sum l adds them before
// that): at most 2^-8 (bf16) or 2^-11 (f16) of each key's probability, averaged over the keys.
template <bool BF16, int D, int RT>
__global__ __launch_bounds__(kWaves * 64, D == 256 ? 1 : 2) void prefix_attn_kernel(PrefixArgs a) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    // Consecutive workgroups go to the XCDs in turn: the blocks of rows that read the
    // same keys sit 8 apart, on one XCD.  The kind whose workgroups take longer comes first.
    const uint32_t group = blockIdx.x >> 3, x = blockIdx.x & 7;
    const uint32_t before = a.own_first ? a.own_groups : a.prefix_groups, i = group < before ? group : group - before;
    if ((group < before) == (a.own_first != 0)) {
        const uint32_t id = i / (uint32_t)a.RO * 8 + x;
        if (id < (uint32_t)a.B * a.Hkv * a.SO) own_work<BF16, D, RT>(a, id, i % (uint32_t)a.RO, smem);
    } else {
        const uint32_t unit = i / (uint32_t)a.RB * 8 + x;
        if (unit < (uint32_t)a.Hkv * a.SP) prefix_work<BF16, D>(a, unit, i % (uint32_t)a.RB, smem);
    }
}

// Joins a row's parts: o = sum 2^(m_s - top) o_s / sum 2^(m_s - top) l_s, in part order.
// W waves per row: with four, wave w adds parts w, w + 4, .. and the four sums are added in wave order.
template <bool BF16, int D, int W>
__global__ __launch_bounds__(256) void prefix_merge_kernel(PrefixArgs a) {
    constexpr int C = D / 64;   // columns per lane
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave % W;
    const size_t row = (size_t)blockIdx.x * (4 / W) + wave / W, rows = (size_t)a.B * a.T * a.Hq;
    const bool there = row < rows;
    float v[C], sum = 0.f, top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = 0.f;
    if (there) {
        const float* const src = a.part_o + row * a.parts * D + lane * C;
        constexpr int H = kMaxParts / 64;   // a lane's parts: lane, lane + 64, ..
        float2 ml[H];
#pragma unroll
        for (int k = 0; k < H; ++k) {
            ml[k] = float2{-__builtin_inff(), 0.f};
            if (lane + 64 * k < a.parts) ml[k] = a.part_ml[row * a.parts + lane + 64 * k];
        }
        float x[8][C];
        auto fetch = [&](int s0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int s = min(s0 + W * j, a.parts - 1);   // past the end: a part that is not added
#pragma unroll
                for (int i = 0; i < C; ++i) x[j][i] = src[(size_t)s * D + i];
            }
        };
        fetch(w);
#pragma unroll
        for (int k = 0; k < H; ++k) top = __builtin_fmaxf(top, ml[k].x);
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, s));
        float f[H];
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < H; ++k) f[k] = weight_of(ml[k].x, top), sum += f[k] * ml[k].y;
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
        for (int s0 = w; s0 < a.parts; s0 += 8 * W) {
            if (s0 != w) fetch(s0);
            float fh = f[0];   // the eight parts lie in one of the blocks of 64
#pragma unroll
            for (int k = 1; k < H; ++k) fh = s0 >= 64 * k ? f[k] : fh;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int s = s0 + W * j;
                const float fs = bitcast<float>(__builtin_amdgcn_readlane(bitcast<int>(fh), s & 63));
#pragma unroll
                for (int i = 0; i < C; ++i) v[i] = s < a.parts ? __builtin_fmaf(fs, x[j][i], v[i]) : v[i];
            }
        }
    }
    if constexpr (W > 1) {
        __shared__ float parts[4][D];
#pragma unroll
        for (int i = 0; i < C; ++i) parts[wave][lane * C + i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C; ++i) {
            v[i] = parts[0][lane * C + i];
#pragma unroll
            for (int k = 1; k < 4; ++k) v[i] += parts[k][lane * C + i];
        }
    }
    if (!there || w != 0) return;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < C; ++i) odd |= v[i] != v[i];
    if (odd && sum - sum == 0.f) settle<BF16, C>(a, row / (uint32_t)a.Hq, (uint32_t)(row % (uint32_t)a.Hq) / (uint32_t)a.G, lane * C, v);
    const float f = sum == 0.f ? 0.f : 1.0f / sum;
    uint16_t* const to = a.out + row * D + lane * C;
    if constexpr (C == 1) {
        *to = (uint16_t)pack2<BF16>(v[0] * f, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < C; i += 2) *(uint32_t*)(to + i) = pack2<BF16>(v[i] * f, v[i + 1] * f);
    }
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -__builtin_inff() : (top - kLift<BF16> + __builtin_log2f(sum)) * kLn2;
}

typedef void (*kernel_t)(PrefixArgs);

template <bool BF16, int D>
kernel_t attend(int rt) {
    return rt == 1 ? prefix_attn_kernel<BF16, D, 1> : prefix_attn_kernel<BF16, D, 2>;
}
template <bool BF16>
kernel_t attend(int D, int rt) {
    return D == 64 ? attend<BF16, 64>(rt) : D == 128 ? attend<BF16, 128>(rt) : prefix_attn_kernel<BF16, 256, 1>;
}
template <bool BF16, int D>
kernel_t merge(int w) {
    return w == 1 ? prefix_merge_kernel<BF16, D, 1> : prefix_merge_kernel<BF16, D, 4>;
}
template <bool BF16>
kernel_t merge(int D, int w) {
    return D == 64 ? merge<BF16, 64>(w) : D == 128 ? merge<BF16, 128>(w) : merge<BF16, 256>(w);
}

// The kernels' dynamic LDS passes the default limit: said once per process and device.
void allow_lds() {
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices || done[dev].load(std::memory_order_acquire)) return;
    for (int D : {64, 128, 256})
        for (int rt : {1, 2})
            for (kernel_t k : {attend<false>(D, rt), attend<true>(D, rt)})
                (void)hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicLds);
    done[dev].store(true, std::memory_order_release);
}

size_t lds_bytes(int D, int rt, bool shared) {
    const size_t ring = shared ? (size_t)kStages * 2 * kTile * D * 2 : 0;
    const size_t join = (size_t)kWaves * 16 * rt * (D + 6) * sizeof(float);
    return ring > join ? ring : join;
}

struct Plan {
    int SP, SO, RB, RO, rt;
    int run;                  // requests of a launch
    long long prefix_groups, own_groups;
    bool own_first;
    bool ok;
};

// The form and the splits of the keys with the least estimated time: workgroups
// of both kinds fill the GPU's places, each a start and a number of steps (measured on
// MI355X, a workgroup beside another one on its CU), the longer kind first; and no less than the bytes take.
Plan make_plan(int B, int T, int Hq, int Hkv, int D, int max_prefix, int max_len) {
    const double kStart = 4.0, kMerge = 4.0, kBytesPerUs = 5.5e6, kPartBytesPerUs = 4.5e6;
    const double own_step = D == 64 ? 0.9 : D == 128 ? 2.2 : 3.5, prefix_step = D == 64 ? 0.7 : D == 128 ? 1.15 : 1.6;
    // Heads of 256 start late (a block of rows for itself on a CU, nothing beside it).  Six batches of 1 to 128 requests behind 100
    // to 32768 keys, both forms measured: the faster one is taken, but for two of the 42 (6 requests of 7 drafts
    // behind 8192 keys: shared 30 us, each for itself 26; 128 of 2 behind 682: 25 and 22).
    const double prefix_start = D == 256 ? 11.0 : kStart;
    const int G = Hq / Hkv, R = T * G;
    const long long places = (long long)w4h::cu_count() * (D == 256 ? 1 : 2);
    const long long ptiles = ((long long)max_prefix + kTile - 1) / kTile, otiles = ((long long)max_len + T + kTile - 1) / kTile;
    const bool in_l2 = ptiles * kTile * Hkv * D * 4 <= (32LL << 20);
    Plan best{};
    double least = 0;
    // A prefix of one tile is not worth its parts (1024 requests of 32/4 heads of 256, 100 of their own: shared 161 us, read
    // again by each 129; 4096 of 40/8 heads of 64: 258 and 204; 1024 of 8 heads of 256 without a context: 170 and 175).
    for (int shared = 0; shared <= (max_prefix > kTile ? 1 : 0); ++shared) {
        const int rt = R <= 16 || D == 256 ? 1 : 2, RO = (R + 16 * rt - 1) / (16 * rt);
        const long long units = (long long)B * Hkv * RO, blocks = (long long)Hkv * (((long long)B * R + kBlockRows - 1) / kBlockRows);
        // Splits worth a look: a few, and those that fill the places once, or what the other kind leaves of them.
        const long long left = places > units ? (places - units) / blocks : 0;
        for (long long SP : {1LL, 2LL, 3LL, 4LL, 6LL, 8LL, 12LL, 16LL, 24LL, 32LL, 48LL, 64LL, 96LL, 128LL, 192LL, places / blocks, left}) {
            if (!shared && SP != 1) continue;
            if (SP > 48 && SP * blocks > places) continue;   // many parts only where they fill the places once
            if (shared && (SP < 1 || SP >= kMaxParts || (SP > 1 && SP * 4 > ptiles))) continue;
            for (long long SO : {1LL, 2LL, 3LL, 4LL, 6LL, 8LL, 12LL, 16LL, 32LL, 64LL, 128LL, places / units}) {
                if (SO > 64 && SO * units > places) continue;
                Plan p{};
                p.SP = shared ? (int)SP : 0, p.SO = (int)SO, p.rt = rt, p.RO = RO;
                const long long tiles = otiles + (shared ? 0 : ptiles);
                const int parts = p.SP + p.SO;
                if (SO < 1 || parts > kMaxParts || (SO > 1 && SO * 2 * kWaves > tiles)) continue;
                // Requests of a run: their parts stay below the limit.
                const long long row = parts > 1 ? (long long)T * Hq * parts * (D + 2) * 4 : 0;
                if (row > (long long)kMaxPartBytes) continue;
                long long run = row ? (long long)kMaxPartBytes / row : B;
                run = run < 1 ? 1 : run < B ? run : B;
                const long long runs = (B + run - 1) / run;
                p.run = (int)((B + runs - 1) / runs);
                p.RB = (int)(((long long)p.run * R + kBlockRows - 1) / kBlockRows);
                p.prefix_groups = ((long long)Hkv * p.SP + 7) / 8 * p.RB;
                p.own_groups = ((long long)p.run * Hkv * SO + 7) / 8 * p.RO;
                const long long merge_rows = (long long)p.run * T * Hq;
                if ((p.prefix_groups + p.own_groups) * 8 * 256 > kMaxLanes || (parts > 1 && merge_rows * 256 > kMaxLanes)) continue;
                const double np = (double)Hkv * p.SP * p.RB, no = (double)p.run * Hkv * SO * p.RO;
                const double dp = shared ? prefix_start + ceil((double)ptiles / SP) * prefix_step : 0;
                const double turns = (double)tiles / SO / kWaves, dn = kStart + 0.5 * (turns + ceil(turns)) * own_step * p.rt;
                p.own_first = dn > dp;
                // The longer kind in whole rounds, the shorter one in the places that are left.
                const double nl = p.own_first ? no : np, dl = p.own_first ? dn : dp, work = (np * dp + no * dn) / places;
                const double rounds = ceil(nl / places) * dl;
                double time = work > rounds ? work + 0.25 * (p.own_first ? dp : dn) : rounds;
                const double again = 1 + (p.run - 1) * (in_l2 ? 0.1 : 0.8);   // readings of a prefix that is not shared
                const double bytes = ((double)ptiles * (shared ? 1 : again) + (double)otiles * p.run) * kTile * Hkv * D * 4;
                if (time < bytes / kBytesPerUs) time = bytes / kBytesPerUs + 0.1 * dl;
                if (parts > 1) time += kMerge + (double)merge_rows * parts * D * 4 / kPartBytesPerUs;
                time *= runs;
                if (!best.ok || time < least) best = p, best.ok = true, least = time;
            }
        }
    }
    return best;
}

// The workspace that is asked for: the most that the plans of this shape or of any smaller one (fewer requests, drafts,
// shorter lengths) can take, since fewer requests take more parts.  The largest batch's workspace then serves all.
size_t workspace_of(int B, int T, int Hq, int D, int max_prefix, int max_len) {
    const long long ptiles = ((long long)max_prefix + kTile - 1) / kTile, tiles = ((long long)max_len + T + kTile - 1) / kTile + ptiles;
    const long long SP = max_prefix > kTile ? (ptiles / 4 < 1 ? 1 : ptiles / 4) : 0, SO = tiles / (2 * kWaves) < 1 ? 1 : tiles / (2 * kWaves);
    const long long parts = SP + SO < kMaxParts ? SP + SO : kMaxParts;
    if (parts == 1) return 0;
    const long long bytes = (long long)B * T * Hq * parts * (D + 2) * 4;
    return w4h::ws_bytes(bytes < (long long)kMaxPartBytes ? (size_t)bytes : kMaxPartBytes);
}

int check_shape(int B, int T, int Hq, int Hkv, int D, int max_prefix, int max_len) {
    if (B < 1 || T < 1 || T > 64 || Hkv < 1 || Hq < Hkv || Hq % Hkv || max_len < 0 || max_len > (1 << 30) || max_prefix < 0 ||
        max_prefix > (1 << 30))
        return W4A16_ERR_SHAPE;
    if (Hq > (1 << 16) || (long long)B * Hq > (1LL << 24)) return W4A16_ERR_SHAPE;
    if (D != 64 && D != 128 && D != 256) return W4A16_ERR_UNSUPPORTED;
    return W4A16_OK;
}

}  // namespace

extern "C" int prefix_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int max_prefix, int max_len,
                                           size_t* bytes) {
    if (!bytes) return W4A16_ERR_NULL;
    if (int rc = check_shape(B, T, Hq, Hkv, D, max_prefix, max_len)) return rc;
    const Plan p = make_plan(B, T, Hq, Hkv, D, max_prefix, max_len);
    if (!p.ok) return W4A16_ERR_UNSUPPORTED;
    *bytes = workspace_of(B, T, Hq, D, max_prefix, max_len);
    return W4A16_OK;
}

extern "C" int prefix_attn(const void* q, long long q_stride, const void* k, const void* v, int dtype, int num_pages,
                           int page_size, long long page_stride, long long token_stride, long long head_stride,
                           const int32_t* prefix_table, const int32_t* prefix_len, int max_prefix,
                           const int32_t* block_table, int table_stride, const int32_t* lens, int max_len,
                           const uint64_t* tree_mask, float scale, void* out, float* lse, int B, int T, int Hq, int Hkv,
                           int D, void* workspace, size_t workspace_bytes, w4a16_stream_t stream) {
    if (!q || !k || !v || !prefix_len || !block_table || !lens || !tree_mask || !out) return W4A16_ERR_NULL;
    if (dtype != W4A16_F16 && dtype != W4A16_BF16) return W4A16_ERR_DTYPE;
    if (int rc = check_shape(B, T, Hq, Hkv, D, max_prefix, max_len)) return rc;
    if (max_prefix > 0 && !prefix_table) return W4A16_ERR_NULL;
    if (num_pages < 1 || page_size < 1 || (page_size & (page_size - 1)) || table_stride < 1 ||
        (long long)table_stride * page_size < (long long)max_len + T)
        return W4A16_ERR_SHAPE;
    if (q_stride < (long long)Hq * D || q_stride % 8 || page_stride < 0 || token_stride < 0 || head_stride < 0 ||
        (unsigned long long)page_size * (unsigned long long)token_stride >= (1ull << 30) || page_stride % 8 ||
        token_stride % 8 || head_stride % 8 || !(scale == scale) || scale - scale != 0.f)
        return W4A16_ERR_SHAPE;
    for (const void* p : {q, k, v, (const void*)out, (const void*)workspace})
        if (!w4h::aligned16(p)) return W4A16_ERR_ALIGN;
    if (((uintptr_t)prefix_table & 3) || ((uintptr_t)prefix_len & 3) || ((uintptr_t)lens & 3) || ((uintptr_t)block_table & 3) ||
        ((uintptr_t)tree_mask & 7) || ((uintptr_t)lse & 3))
        return W4A16_ERR_ALIGN;
    if (page_size < 16) return W4A16_ERR_UNSUPPORTED;   // a half of a tile lies in one page
    const Plan p = make_plan(B, T, Hq, Hkv, D, max_prefix, max_len);
    if (!p.ok) return W4A16_ERR_UNSUPPORTED;
    const size_t need = workspace_of(B, T, Hq, D, max_prefix, max_len);
    if (need && !workspace) return W4A16_ERR_NULL;
    if (workspace_bytes < need) return W4A16_ERR_WORKSPACE;
    PrefixArgs a{};
    a.k = (const uint16_t*)k, a.v = (const uint16_t*)v;
    a.prefix_table = prefix_table, a.prefix_len = prefix_len;
    a.q_stride = q_stride, a.page_stride = page_stride, a.token_stride = token_stride, a.head_stride = head_stride;
    a.num_pages = num_pages, a.table_stride = table_stride, a.max_prefix = max_prefix, a.max_len = max_len;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.scale2 = fmaxf(fabsf(scale) * kLog2e, 0x1p-126f);   // not 0: -inf marks what a row does not see
    a.q_sign = scale < 0.f ? 0x80008000u : 0u;
    a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv;
    a.SP = p.SP, a.SO = p.SO, a.RO = p.RO, a.parts = p.SP + p.SO, a.own_first = p.own_first;
    const bool bf16 = dtype == W4A16_BF16;
    const hipStream_t st = (hipStream_t)stream;
    const size_t lds = lds_bytes(D, p.rt, p.SP > 0);
    allow_lds();
    w4h::begin_launches();
    for (int b0 = 0; b0 < B; b0 += p.run) {
        const size_t tok = (size_t)b0 * T;
        a.B = B - b0 < p.run ? B - b0 : p.run;
        a.RB = (int)(((long long)a.B * T * a.G + kBlockRows - 1) / kBlockRows);
        a.prefix_groups = (uint32_t)(((long long)Hkv * p.SP + 7) / 8 * a.RB);
        a.own_groups = (uint32_t)(((long long)a.B * Hkv * p.SO + 7) / 8 * a.RO);
        a.q = (const uint16_t*)q + tok * q_stride, a.table = block_table + (size_t)b0 * table_stride;
        a.lens = lens + b0, a.mask = tree_mask + tok;
        a.out = (uint16_t*)out + tok * Hq * D, a.lse = lse ? lse + tok * Hq : nullptr;
        const size_t rows = (size_t)a.B * T * Hq;
        a.part_o = (float*)w4h::ws_part(workspace);
        a.part_ml = workspace ? (float2*)(a.part_o + rows * a.parts * D) : nullptr;
        hipLaunchKernelGGL(bf16 ? attend<true>(D, p.rt) : attend<false>(D, p.rt), dim3((a.prefix_groups + a.own_groups) * 8), dim3(kWaves * 64), lds,
                           st, a);
        if (a.parts > 1) {
            // Four waves join a row where few rows have many parts (320 of 57: 4.8 us, a wave each 6.8; 3584 of 13: 7.8 and 6.7).
            const int w = rows * 4 < 16384 && a.parts > 16 ? 4 : 1;
            hipLaunchKernelGGL(bf16 ? merge<true>(D, w) : merge<false>(D, w), dim3((unsigned)((rows * w + 3) / 4)), dim3(256), 0, st, a);
        }
    }
    w4h::note_variant("%s D=%lld prefix_splits=%lld own_splits=%lld row_tiles=%lld requests=%lld of %lld", "prefix_attn", D, p.SP, p.SO, p.rt, p.run, B);
    return w4h::launch_status();
}
