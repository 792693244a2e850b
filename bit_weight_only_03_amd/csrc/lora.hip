// lora.hip -- low-rank adapters of many requests beside a shared projection:
// y = base + s B (A x), each row with an adapter of its own.
//
// Rows come in tiles of 16 (64 in the first product of many rows), and the distinct
// adapters of a tile are taken in turn.  One MFMA covers 16 rows, so an adapter's A
// and B are read once for all its rows there; rows of other adapters enter as zeros
// (their x is not fetched) and their results are not stored.  First product: h^T = A x^T,
// rank by rows, K divided among the waves, whose sums are added in LDS in wave order.
// Second: y = h B^T, 128 columns at a time: lane c of a row of 16 takes columns 8 c ..
// 8 c + 7, so that base and y move in runs of 256 bytes.
//
// What the matrix unit wants in a lane (16 bytes of a row, the rows side by side in the
// lanes) is not what the caches like (the lanes side by side in a row): loaded like
// that, an instruction takes 32 accesses of the CU's cache for 1 KiB instead of 16 or less.  So A,
// B and the x of many rows go through LDS, whole lines at a time, in a ring that each wave
// has for itself: no barriers, only counted waits.
//
// Few rows are bound by latency (one token through qkv 5120 -> 7168, rank 16: 8.2 us in a graph; what it
// reads takes 0.2) and by reading the adapters (64 requests of 48 adapters through gate/up 5120 ->
// 34816, ranks 8 to 32: 32 us, 2.2 TB/s of 69 MB, and padded ranks are read too); many rows by moving x, base and y (4096 rows
// through qkv, rank 16, in 54 us, 3.0 TB/s: two launches, of which the first reads x at what the L2s give).
// Times are per call with three sets of inputs in turn; the same inputs again, from the caches, take 27 and 42 us.
#include "attn_common.h"
#include "../../include/lora.h"

using namespace w4k;

namespace {

constexpr int kRows = 16;              // rows of a tile
constexpr int kMaxR = 256;
constexpr int kGroup = 128;            // columns that a wave takes at a time
constexpr int kUnit = 64;              // k that a wave takes at a time: a line of each row
constexpr int kStep = 32;              // ranks of B at a time
constexpr int kStepBytes = kGroup * kStep * 2;
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
    int n, M, N, K, R, parts;
    int part_start[LORA_MAX_PARTS + 1];
    int block_start[LORA_MAX_PARTS + 1];   // first column block of each part
    int cols;             // columns of a block, a multiple of 64
    int turns, first_turns;   // workgroups that share a tile's adapters
    uint32_t first_tiles; // row tiles of the first launch, which may be larger
    int first_groups;     // of 16 RK rows of a
    int run;              // row tiles of a workgroup of the second launch of many rows
    int slices;           // slices of K (1 where the products are one launch)
};

// A tile's rows that share one adapter.
struct Rows {
    int m0;          // the tile's first row
    int id;          // adapter, -1: none
    int ranks;       // the adapter's
    int rank;        // rounded up to a multiple of 8: what is read of it
    float scale;
    uint64_t members;
};

// Stages of the first product's ring: 16 to 20 KiB for each of eight waves, 28 to 36 for each of four (MT = 4).
constexpr int first_stages(int rk, int mt) { return mt == 1 ? (rk == 1 ? 4 : rk == 2 ? 3 : 2) : rk <= 2 ? 3 : 2; }
constexpr int first_stage_bytes(int rk, int mt) { return 2048 * (rk + mt); }
constexpr size_t first_lds(int rk, int mt, int waves) {
    const size_t ring = (size_t)waves * first_stages(rk, mt) * first_stage_bytes(rk, mt), sums = (size_t)waves * rk * mt * 1024;
    return ring > sums ? ring : sums;
}

// 16 RK rows of a (the parts' ranks one after another, from j0 on) times 16 MT rows of x for
// units [u0, u1) of this wave: acc[t MT + m][i] of lane (c, g) is row j0 + 16 t + 4 g + i of a, row 16 m + c of x.
// Loops are not unrolled: a call of few rows passes through this code once, and waits
// for its instructions from L2 (unrolled over the ring, one token took 2 us longer).
template <bool BF16, int RK, int MT>
__device__ __forceinline__ void first_product(const LoraArgs& a, const Rows& r, int j0, int j1, int u0, int u1, uint8_t* ring, float4_t* acc) {
    constexpr int D = first_stages(RK, MT), kStage = first_stage_bytes(RK, MT);
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = 2u * a.K, ranks = (uint32_t)a.parts * a.R;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.a + (size_t)r.id * ranks * a.K, ranks * row_bytes);
    const int last = min(kRows * MT, a.M - r.m0) - 1;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)r.m0 * a.ldx, (uint32_t)(last * a.ldx + a.K) * 2u);
    // Load i of a tile takes its rows 8 i .. 8 i + 7, eight lanes each; chunk p ^ (row % 8) of a row goes to place p.
    const int row8 = lane >> 3;
    const uint32_t chunk = 16u * ((lane & 7) ^ row8);
    uint32_t a_row[2 * RK], x_row[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * RK; ++i) {
        const int j = j0 + 8 * i + row8;
        a_row[i] = j < j1 && (int)((uint32_t)j % (uint32_t)a.R) < r.rank ? (uint32_t)j * row_bytes + chunk : kNowhere;
    }
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) x_row[i] = (r.members >> (8 * i + row8)) & 1u ? (uint32_t)((8 * i + row8) * a.ldx * 2) + chunk : kNowhere;
    const uint32_t end = 2u * min(a.K, u1 * kUnit);
    auto load = [&](int at, int u) {
        const uint32_t k = 2u * (u * kUnit);
        uint8_t* const to = ring + at;
        const bool there = k + chunk < end;
#pragma unroll
        for (int i = 0; i < 2 * RK; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(to + 1024 * i), 16, there ? a_row[i] + k : kNowhere, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(to + 2048 * RK + 1024 * i), 16, there ? x_row[i] + k : kNowhere, 0, 0, 0);
    };
#pragma unroll 1
    for (int i = 0; i < D; ++i) load(i * kStage, u0 + i);
    int at = 0;
#pragma unroll 1
    for (int u = u0; u < u1; ++u) {
        wait_loads<(D - 1) * 2 * (RK + MT)>();
        const uint8_t* const from = ring + at + c * 128;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = 16 * ((4 * s + g) ^ (c & 7));
            u32x4_t w[RK];
#pragma unroll
            for (int t = 0; t < RK; ++t) w[t] = *(const u32x4_t*)(from + 2048 * t + k);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const u32x4_t x = *(const u32x4_t*)(from + 2048 * (RK + m) + k);
#pragma unroll
                for (int t = 0; t < RK; ++t) acc[t * MT + m] = mfma<BF16>(w[t], x, acc[t * MT + m]);
            }
        }
        wait_loads<63>();   // its LDS reads
        load(at, u + D);
        at = at + kStage < D * kStage ? at + kStage : 0;
    }
    wait_loads<0>();
}

// The sums of rows [j0, j1) of a over units [u0, u1), the waves' parts added in wave order:
// put(row of the tile, row of a, four sums).  lds: first_lds(RK, MT, waves) bytes.
template <bool BF16, int RK, int MT, typename F>
__device__ __forceinline__ void sum_h(const LoraArgs& a, const Rows& r, int j0, int j1, int u0, int u1, uint8_t* lds, F put) {
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), waves = blockDim.x >> 6;
    float* const sums = (float*)lds;
    for (; j0 < j1; j0 += 16 * RK) {
        float4_t acc[RK * MT];
#pragma unroll
        for (int i = 0; i < RK * MT; ++i) acc[i] = float4_t{0.f, 0.f, 0.f, 0.f};
#ifdef __HIP_DEVICE_COMPILE__   // the compiler's host pass finds no match for the call
        first_product<BF16, RK, MT>(a, r, j0, j1, u0 + (u1 - u0) * wave / waves, u0 + (u1 - u0) * (wave + 1) / waves, lds + wave * first_stages(RK, MT) * first_stage_bytes(RK, MT), acc);
#endif
        __syncthreads();   // the sums lie where the rings did
#pragma unroll
        for (int i = 0; i < RK * MT; ++i) *(float4_t*)(sums + ((wave * RK * MT + i) * 64 + lane) * 4) = acc[i];
        __syncthreads();
        for (int e = t; e < RK * MT * 64; e += blockDim.x) {
            float4_t v = *(const float4_t*)(sums + e * 4);
#pragma unroll 4
            for (int w = 1; w < waves; ++w) v += *(const float4_t*)(sums + (w * RK * MT * 64 + e) * 4);
            const int j = j0 + 16 * (e / (64 * MT)) + 4 * ((e >> 4) & 3);
            if (j < j1) put((e / 64 % MT) * 16 + (e & 15), j, v);
        }
        __syncthreads();
    }
}

__device__ __forceinline__ bool finite(float v) { return (bitcast<uint32_t>(v) & 0x7f800000u) != 0x7f800000u; }

// fp16 has neither fp32's range nor a third term's use: each row is taken times a power of
// two that brings its largest element to 2^13.  top: the largest finite magnitude's bits
// among this lane's elements; the 16 lanes of a DPP row hold a row.  Returns that power; back takes it back.
__device__ __forceinline__ float to_range(uint32_t top, float& back) {
    top = max(top, dpp<0xB1>(top));
    top = max(top, dpp<0x4E>(top));
    top = max(top, dpp<0x141>(top));
    top = max(top, dpp<0x140>(top));
    const int e = max((int)(top >> 23), 40);                      // biased; below 2^-87 all the same
    back = bitcast<float>((uint32_t)(e - 13) << 23);
    return bitcast<float>((uint32_t)(127 + 127 + 13 - e) << 23);  // 2^(13 - (e - 127)); e <= 254: at least 2^-114
}
__device__ __forceinline__ uint32_t magnitude(float v) { return finite(v) ? bitcast<uint32_t>(v) & 0x7fffffffu : 0u; }

// v as a sum of NT terms of the dtype, two neighbours in a dword.  bf16 terms are cut
// off (a finite value stays finite), the last one is rounded.
template <bool BF16, int NT>
__device__ __forceinline__ void terms_of(float v0, float v1, uint32_t* term) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if constexpr (BF16)
            term[n] = n == NT - 1 ? pk_bf16(v0, v1) : (bitcast<uint32_t>(v0) >> 16) | (bitcast<uint32_t>(v1) & 0xffff0000u);
        else
            term[n] = pk_f16(v0, v1);
        const float t0 = BF16 ? bitcast<float>(term[n] << 16) : f16_bits_to_f32((uint16_t)term[n]);
        const float t1 = BF16 ? bitcast<float>(term[n] & 0xffff0000u) : f16_bits_to_f32((uint16_t)(term[n] >> 16));
        v0 = finite(t0) ? v0 - t0 : 0.f, v1 = finite(t1) ? v1 - t1 : 0.f;
    }
}

// s h in NT terms of the dtype: hb [term][16][stride], ranks past the adapter's are zeros (a row with an
// infinity has NaN there, of the infinity times the zeros that fill a's rank up to eight).
template <bool BF16, int NT>
__device__ __forceinline__ void split_h(const LoraArgs& a, const Rows& r, const float* hf, uint16_t* hb, int stride, float* back) {
    const int row = threadIdx.x >> 4, l = threadIdx.x & 15;
    if (row < kRows) {
        const float* const src = hf + row * (a.R + 4);
        float up = 1.f;
        if constexpr (!BF16) {
            uint32_t top = 0;
            for (int j = l; j < r.ranks; j += 16) top = max(top, magnitude(src[j] * r.scale));
            float down;
            up = to_range(top, down);
            if (l == 0) back[row] = down;
        }
        for (int j = 2 * l; j < stride - 8; j += 32) {
            uint32_t term[NT];
            terms_of<BF16, NT>(j < r.ranks ? src[j] * r.scale * up : 0.f, j + 1 < r.ranks ? src[j + 1] * r.scale * up : 0.f, term);
#pragma unroll
            for (int n = 0; n < NT; ++n) *(uint32_t*)(hb + (n * kRows + row) * stride + j) = term[n];
        }
    }
    __syncthreads();
}

// Calls f for this workgroup's share of the distinct adapters of a tile.
template <int ROWS, typename F>
__device__ __forceinline__ void each_adapter(const LoraArgs& a, int tile, int turn, int turns, bool with_none, F f) {
    const int lane = threadIdx.x & 63, m0 = tile * ROWS;
    const bool there = lane < ROWS && m0 + lane < a.M;
    int id = there ? a.adapter[m0 + lane] : -1;
    // The first 64 adapters' ranks and scales beside the rows' adapters, not after them.
    const int rank64 = a.ranks && lane < a.n ? a.ranks[lane] : a.R;
    const float scale64 = a.scales && lane < a.n ? a.scales[lane] : 1.f;
    id = id < 0 || id >= a.n ? -1 : id;
    uint64_t left = __builtin_amdgcn_ballot_w64(there && (id >= 0 || with_none));
    for (int i = 0; left; ++i) {
        const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t same = __builtin_amdgcn_ballot_w64(there && id == one);
        left &= ~same;
        if (i % turns != turn) continue;
        Rows r{m0, one, 0, 0, 1.f, same};
        if (one >= 0) {
            int rank = __builtin_amdgcn_readlane(rank64, one & 63);
            r.scale = bitcast<float>(__builtin_amdgcn_readlane(bitcast<int>(scale64), one & 63));
            if (one > 63) {
                rank = a.ranks ? a.ranks[one] : a.R;
                r.scale = a.scales ? a.scales[one] : 1.f;
            }
            r.ranks = min(max(__builtin_amdgcn_readfirstlane(rank), 0), a.R);
            r.rank = (r.ranks + 7) & ~7;
        }
        f(r);
    }
}

// Consecutive workgroups go to the XCDs in turn.  Of many rows each XCD takes a run (of n
// workgroups, a multiple of eight), whose adapters then stay in its L2.
__device__ __forceinline__ uint32_t run_of_rows(uint32_t i, uint32_t n) { return i % 8 * (n / 8) + i / 8; }

// Stages of the second product's ring, 8 KiB each, for each of four waves (three leave no room for a second workgroup on the CU).
constexpr int kSecondStages = 2;

// y of columns [n0, n1) of a tile's rows, Y its type.  make_h() leaves s h in hb (and back); the first
// loads are on their way meanwhile.  Rows and columns that are not there are past
// their buffer's end, so that no load or store has a branch around it.
template <bool BF16, int NT, int Y>
struct Second {
    static constexpr int kSize = Y == W4A16_F32 ? 4 : 2, kWords = Y == W4A16_F32 ? 2 : 1;   // bytes of an element, 16 bytes of eight
    static constexpr int kMoves = 4 * kWords;                                               // loads of a base, stores of a result
    const LoraArgs& a;
    const Rows& r;
    int n0, n1;
    int lane, wave, step, c, g;
    uint32_t row_bytes, y_row[4], b_row[2];
    __amdgpu_buffer_rsrc_t ry, rbase;
    const uint16_t* b;

    __device__ __forceinline__ Second(const LoraArgs& a, const Rows& r, int n0, int n1) : a(a), r(r), n0(n0), n1(n1) {
        lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        step = __builtin_amdgcn_readfirstlane(kGroup * (blockDim.x >> 6)), c = lane & 15, g = lane >> 4;
        row_bytes = 2u * a.R;
        const int rows = min(kRows, a.M - r.m0);
        const uint32_t bytes = (uint32_t)((rows - 1) * a.ldy + a.N) * kSize;
        const size_t at = (size_t)r.m0 * a.ldy * kSize;
        ry = make_rsrc((uint8_t*)a.y + at, bytes), rbase = make_rsrc((const uint8_t*)a.base + at, a.base ? bytes : 0u);
        // Lane (c, g) has rows 4 g + i and columns 8 c .. 8 c + 7 of a group.
#pragma unroll
        for (int i = 0; i < 4; ++i) y_row[i] = (r.members >> (4 * g + i)) & 1u ? (uint32_t)((4 * g + i) * a.ldy + 8 * c) * kSize : kNowhere;
        b = a.b + (size_t)max(r.id, 0) * a.N * a.R;
        // Load j of a step fills places 16 j .. 16 j + 15, four lanes each.  Column q has place q ^ (q / 8 % 4), and there
        // chunk p of its 32 ranks lies at p ^ (q / 32): lane (c, g)'s reads of columns 8 c + t are spread over all banks.
#pragma unroll
        for (int j = 0; j < 2; ++j) b_row[j] = (uint32_t)((lane >> 2) ^ (2 * j + (lane >> 5))) * row_bytes;
    }
    __device__ __forceinline__ uint32_t place(int n, int i) const { return n + 8 * c < n1 ? y_row[i] + (uint32_t)n * kSize : kNowhere; }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t columns(int n) const {
        const uint32_t bytes = __builtin_amdgcn_readfirstlane(min(kGroup, max(n1 - n, 0)) * row_bytes);
        return make_rsrc(b + (size_t)__builtin_amdgcn_readfirstlane(min(n, n1)) * a.R, bytes);
    }
    // Ranks 32 s .. of a group's b to LDS.
    __device__ __forceinline__ void load_b(uint8_t* to, int n, int s) const {
        const __amdgpu_buffer_rsrc_t rb = columns(n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t chunk = 16u * ((lane & 3) ^ (j >> 1)) + 64u * s;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(to + 1024 * j), 16, chunk < 2u * r.rank ? 16 * j * row_bytes + b_row[j & 1] + chunk : kNowhere, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void load_base(u32x4_t (*base)[kWords], int n) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < kWords; ++e) base[i][e] = bitcast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(rbase, place(n, i), 16 * e, 0));
    }
    __device__ static __forceinline__ void multiply(const u32x4_t* w, const uint16_t* hb, int stride, int s, float4_t* acc) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int k = NT - 1; k >= 0; --k) {
            const u32x4_t h = *(const u32x4_t*)(hb + (k * kRows + (lane & 15)) * stride + kStep * s + 8 * (lane >> 4));
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[t] = mfma<BF16>(h, w[t], acc[t]);
        }
    }
    // Tile t's column 8 c + t of ranks 8 g .. of the step that lies at `from`.
    __device__ __forceinline__ void read_b(const uint8_t* from, u32x4_t* w) const {
#pragma unroll
        for (int t = 0; t < 8; ++t) w[t] = *(const u32x4_t*)(from + ((8 * c + t) ^ (c & 3)) * (2 * kStep) + 16 * (g ^ (c >> 2)));
    }
    __device__ static __forceinline__ void result(const float4_t* acc, const u32x4_t (*base)[kWords], const float* f, u32x4_t (*out)[kWords]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (Y == W4A16_F32) {
                    v[e] = bitcast<float>(base[i][e >> 2][e & 3]);
                } else {
                    const uint32_t q = base[i][0][e >> 1];
                    v[e] = Y == W4A16_BF16 ? bitcast<float>(e & 1 ? q & 0xffff0000u : q << 16) : f16_bits_to_f32((uint16_t)(e & 1 ? q >> 16 : q));
                }
                v[e] = __builtin_fmaf(acc[e][i], f[i], v[e]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (Y == W4A16_F32) out[i][0][j] = bitcast<uint32_t>(v[j]), out[i][kWords - 1][j] = bitcast<uint32_t>(v[4 + j]);
                else out[i][0][j] = Y == W4A16_BF16 ? pk_bf16(v[2 * j], v[2 * j + 1]) : pk_f16(v[2 * j], v[2 * j + 1]);
            }
        }
    }
    __device__ __forceinline__ void store(const u32x4_t (*out)[kWords], int n) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < kWords; ++e) __builtin_amdgcn_raw_buffer_store_b128(out[i][e], ry, place(n, i), 16 * e, 0);
    }
    // Rows without an adapter: their sum, 0, is taken times -1, as base + 0 would lose the sign of a base of -0.
    __device__ __forceinline__ void scales(const float* back, float* f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = r.id < 0 ? -1.f : BF16 ? 1.f : back[4 * g + i];
    }

    // At most 32 RS ranks, a group or two for a wave: b straight to registers, asked for before h is made.
    template <int RS>
    struct Few {
        u32x4_t w[RS][8], base[4][kWords];
    };
    template <int RS>
    __device__ __forceinline__ void few_load(Few<RS>& q, int n) const {
        const __amdgpu_buffer_rsrc_t rb = columns(n);
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int t = 0; t < 8; ++t)
                q.w[s][t] = bitcast<u32x4_t>(
                    __builtin_amdgcn_raw_buffer_load_b128(rb, kStep * s + 8 * g < r.rank ? (8 * c + t) * row_bytes + 64 * s + 16 * g : kNowhere, 0, 0));
        load_base(q.base, n);
    }
    template <int RS>
    __device__ __forceinline__ void few(Few<RS>& q, const uint16_t* hb, int stride, const float* back) const {
        float f[4];
        scales(back, f);
#pragma unroll 1
        for (int n = n0 + kGroup * wave; n < n1; n += step) {
            u32x4_t out[4][kWords];
            float4_t acc[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < RS; ++s) multiply(q.w[s], hb, stride, s, acc);
            result(acc, q.base, f, out);
            __builtin_amdgcn_sched_barrier(0);
            few_load(q, n + step);
            store(out, n);
        }
    }

    // At most 32 ranks: a ring of groups, and as many bases in registers.
    template <typename F>
    __device__ __forceinline__ void one_step(uint8_t* ring, const uint16_t* hb, int stride, const float* back, F make_h) const {
        constexpr int D = kSecondStages;
        u32x4_t base[D][4][kWords], out[4][kWords];
        int n = n0 + kGroup * wave;
#pragma unroll
        for (int i = 0; i < D; ++i) {
            load_b(ring + i * kStepBytes, n + i * step, 0);
            load_base(base[i], n + i * step);
#pragma unroll
            for (int e = 0; e < kMoves; ++e)   // stores that go nowhere: the loop's counted waits then hold from its start
                __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{0u, 0u, 0u, 0u}, ry, kNowhere, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        make_h();
        float f[4];
        scales(back, f);
#pragma unroll 1
        for (; n < n1; n += D * step) {
#pragma unroll
            for (int i = 0; i < D; ++i) {
                wait_loads<kMoves + (D - 1) * (8 + 2 * kMoves)>();
                u32x4_t w[8];
                read_b(ring + i * kStepBytes, w);
                float4_t acc[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
                multiply(w, hb, stride, 0, acc);
                result(acc, base[i], f, out);
                wait_loads<63>();   // its LDS reads
                __builtin_amdgcn_sched_barrier(0);
                load_b(ring + i * kStepBytes, n + (i + D) * step, 0);
                load_base(base[i], n + (i + D) * step);
                store(out, n + i * step);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        wait_loads<0>();
    }

    // More ranks: a ring of steps of 32.
    template <typename F>
    __device__ __forceinline__ void steps(uint8_t* ring, const uint16_t* hb, int stride, const float* back, F make_h) const {
        constexpr int D = kSecondStages;
        const int steps = max((r.rank + kStep - 1) / kStep, 1);
        int n = n0 + kGroup * wave, ahead_n = n, ahead_s = 0, slot = 0;
        auto next = [&] {   // asks for the step after the last one that was asked for
            load_b(ring + slot * kStepBytes, ahead_n, ahead_s);
            slot = slot + 1 < D ? slot + 1 : 0;
            const bool last = ahead_s + 1 == steps;
            ahead_n += last ? step : 0, ahead_s = last ? 0 : ahead_s + 1;
        };
#pragma unroll
        for (int i = 0; i < D; ++i) next();
        make_h();
        float f[4];
        scales(back, f);
#pragma unroll 1
        for (; n < n1; n += step) {
            u32x4_t base[4][kWords], out[4][kWords];
            load_base(base, n);
            float4_t acc[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int s = 0; s < steps; ++s) {
                wait_loads<(D - 1) * 8>();   // of what came after its own: other steps' loads, 8 each, at least
                u32x4_t w[8];
                read_b(ring + slot * kStepBytes, w);
                multiply(w, hb, stride, s, acc);
                wait_loads<63>();
                __builtin_amdgcn_sched_barrier(0);
                next();
                __builtin_amdgcn_sched_barrier(0);
            }
            result(acc, base, f, out);
            store(out, n);
        }
        wait_loads<0>();
    }
};

// One launch: both products, a workgroup for (tile, turn, column block); the first product is
// made again by each block of columns, from L2.
constexpr int both_waves(int rk) { return rk > 2 ? 4 : 8; }
template <bool BF16, int RK, int Y>
__global__ __launch_bounds__(both_waves(RK) * 64, 2) void lora_both_kernel(LoraArgs a) {
    constexpr int NT = BF16 && Y == W4A16_F32 ? 3 : 2, RS = RK > 2 ? 2 : 1, stride = kStep * RS + 8;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    uint8_t* const ring = smem;
    float* const hf = (float*)(smem + first_lds(RK, 1, both_waves(RK)));   // [16][R + 4]
    float* const back = hf + kRows * (kStep * RS + 4);                     // [16]
    uint16_t* const hb = (uint16_t*)(back + kRows);                   // [NT][16][stride]
    const int blocks = a.block_start[a.parts], block = blockIdx.x % (uint32_t)blocks;
    const uint32_t unit = blockIdx.x / (uint32_t)blocks;
    const int turn = unit % (uint32_t)a.turns, tile = unit / (uint32_t)a.turns, units = (a.K + kUnit - 1) / kUnit;
    int part = 0;
    while (part + 1 < a.parts && block >= a.block_start[part + 1]) ++part;
    const int n0 = a.part_start[part] + (block - a.block_start[part]) * a.cols, n1 = min(n0 + a.cols, a.part_start[part + 1]);
    // base copied for rows without an adapter, unless it is y itself
    each_adapter<kRows>(a, tile, turn, a.turns, a.base != a.y, [&](const Rows& r) {
        const Second<BF16, NT, Y> second(a, r, n0, n1);
        typename Second<BF16, NT, Y>::template Few<RS> q;
        second.few_load(q, n0 + kGroup * second.wave);
        sum_h<BF16, RK, 1>(a, r, part * a.R, part * a.R + r.rank, 0, units, ring, [&](int row, int j, const float4_t& v) {
            *(float4_t*)(hf + row * (a.R + 4) + j - part * a.R) = v;
        });
        split_h<BF16, NT>(a, r, hf, hb, stride, back);
        second.few(q, hb, stride, back);
        __syncthreads();
    });
}

// Two launches, where that costs more: slices of the sums over K, 16 RK rows of the parts' a each ..
template <bool BF16, int RK, int MT>
__global__ __launch_bounds__(MT == 1 ? 512 : 256, 2) void lora_first_kernel(LoraArgs a) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const uint32_t each = gridDim.x / (uint32_t)a.first_turns, turn = blockIdx.x / each, at = blockIdx.x % each;
    const uint32_t id = MT > 1 ? run_of_rows(at, each) : at, tile = id / (uint32_t)(a.slices * a.first_groups);
    const int slice = id % (uint32_t)a.slices, group = id / (uint32_t)a.slices % (uint32_t)a.first_groups, units = (a.K + kUnit - 1) / kUnit, ranks = a.parts * a.R;
    if (tile >= a.first_tiles) return;
    const int j0 = 16 * RK * group, j1 = min(j0 + 16 * RK, ranks);
    const int u0 = units * slice / a.slices, u1 = units * (slice + 1) / a.slices;
    each_adapter<kRows * MT>(a, tile, turn, a.first_turns, false, [&](const Rows& r) {
        float* const dst = a.h + ((size_t)slice * a.M + r.m0) * ranks;
        sum_h<BF16, RK, MT>(a, r, j0, j1, u0, u1, smem, [&](int row, int j, const float4_t& v) {
            if ((r.members >> row) & 1u && (int)((uint32_t)j % (uint32_t)a.R) < r.rank) *(float4_t*)(dst + (size_t)row * ranks + j) = v;
        });
    });
}

// .. and their sums in slice order times B: at most 64 rows, or more than 64 ranks.  RS: ranks in steps of 32.
template <bool BF16, int Y, int RS>
__global__ __launch_bounds__(256, 2) void lora_second_kernel(LoraArgs a) {
    constexpr int NT = BF16 && Y == W4A16_F32 ? 3 : 2, stride = kStep * RS + 8;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int t = threadIdx.x, ranks = a.parts * a.R;
    uint8_t* const ring = smem + (t >> 6) * kSecondStages * kStepBytes;
    float* const hf = (float*)(smem + 4 * kSecondStages * kStepBytes);   // [16][R + 4]
    float* const back = hf + kRows * (kStep * RS + 4);                            // [16]
    uint16_t* const hb = (uint16_t*)(back + kRows);                               // [NT][16][stride]
    const uint32_t blocks = a.block_start[a.parts], unit = blockIdx.x / blocks;
    const int block = blockIdx.x % blocks, turn = unit % (uint32_t)a.turns, tile = unit / (uint32_t)a.turns;
    int part = 0;
    while (part + 1 < a.parts && block >= a.block_start[part + 1]) ++part;
    const int n0 = a.part_start[part] + (block - a.block_start[part]) * a.cols, n1 = min(n0 + a.cols, a.part_start[part + 1]);
    each_adapter<kRows>(a, tile, turn, a.turns, a.base != a.y, [&](const Rows& r) {
        const Second<BF16, NT, Y> second(a, r, n0, n1);
        auto make_h = [&] {
            const float* const src = a.h + (size_t)r.m0 * ranks + part * a.R;
            const size_t step = (size_t)a.M * ranks;
            const int quads = r.rank / 4;
            for (int e = t; e < kRows * quads; e += blockDim.x) {
                const int row = e / quads, j = e % quads * 4;
                float4_t v = {0.f, 0.f, 0.f, 0.f};
                if ((r.members >> row) & 1u) {
                    const float* const p = src + (size_t)row * ranks + j;
                    for (int s = 0; s < a.slices; s += 8) {
                        float4_t x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = *(const float4_t*)(p + min(s + k, a.slices - 1) * step);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (s + k < a.slices) v += x[k];
                    }
                }
                *(float4_t*)(hf + row * (a.R + 4) + j) = v;
            }
            __syncthreads();
            split_h<BF16, NT>(a, r, hf, hb, stride, back);
        };
        if constexpr (RS == 1) second.one_step(ring, hb, stride, back, make_h);
        else second.steps(ring, hb, stride, back, make_h);
        __syncthreads();
    });
}

// The same of more than 64 rows, up to 64 ranks: a workgroup takes 512 columns of a run of row tiles, and every turns-th
// of each tile's adapters.  It makes h of the whole run first; then a wave keeps its 128 columns of
// b in registers for as long as the adapter stays the same, and only base and y move.
template <bool BF16, int Y, int RS>
__global__ __launch_bounds__(256, 2) void lora_rows_kernel(LoraArgs a) {
    constexpr int NT = BF16 && Y == W4A16_F32 ? 3 : 2, stride = kStep * RS + 8, D = 2;
    typedef Second<BF16, NT, Y> S;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    int* const ids = (int*)smem;                            // [run 16]: -1 none, -2 no row
    float* const back = (float*)(ids + a.run * kRows);      // [run 16]
    uint16_t* const hb = (uint16_t*)(back + a.run * kRows); // [run][NT][16][stride]
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), c = lane & 15, g = lane >> 4;
    const uint32_t each = gridDim.x / (uint32_t)a.turns, id = run_of_rows(blockIdx.x % each, each), blocks = a.block_start[a.parts];
    const int turn = blockIdx.x / each, block = id % blocks, first = id / blocks * a.run, tiles = min(a.run, (a.M + kRows - 1) / kRows - first);
    if (tiles <= 0) return;
    int part = 0;
    while (part + 1 < a.parts && block >= a.block_start[part + 1]) ++part;
    const int n = __builtin_amdgcn_readfirstlane(a.part_start[part] + (block - a.block_start[part]) * a.cols + kGroup * wave);
    const int n1 = __builtin_amdgcn_readfirstlane(min(n - kGroup * wave + a.cols, a.part_start[part + 1]));
    // Base and y of a tile.
    auto of_tile = [&](const void* p, int i) {
        const int m0 = (first + i) * kRows, rows = min(kRows, a.M - m0);
        const uint32_t bytes = p && i < tiles ? (uint32_t)((rows - 1) * a.ldy + a.N) * S::kSize : 0u;
        return make_rsrc((const uint8_t*)p + (size_t)m0 * a.ldy * S::kSize, __builtin_amdgcn_readfirstlane(bytes));
    };
    uint32_t at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = n + 8 * c < n1 ? (uint32_t)((4 * g + i) * a.ldy + n + 8 * c) * S::kSize : kNowhere;
    u32x4_t base[D][4][S::kWords];
    auto load_base = [&](int slot, int i) {
        const __amdgpu_buffer_rsrc_t r = of_tile(a.base, i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < S::kWords; ++e) base[slot][k][e] = bitcast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(r, at[k], 16 * e, 0));
    };
#pragma unroll
    for (int i = 0; i < D; ++i) load_base(i, i);

    // h: 16 lanes take a row (four ranks each), the workgroup eight tiles at a time.  The sums
    // are asked for before the rows' adapters, and those with no wait between them.
    const int ranks = a.parts * a.R, l = t & 15;
    constexpr int T = 8;
    for (int i0 = 0; i0 < tiles; i0 += T) {
        int who[T], rank[T];
        float scale[T];
        float4_t v[T];
        auto row_of = [&](int k) { return (first + i0 + k) * kRows + (t >> 4); };
#pragma unroll
        for (int k = 0; k < T; ++k) who[k] = a.adapter[min(row_of(k), a.M - 1)], v[k] = float4_t{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < a.slices; s += 2) {
            float4_t x[T][2];
#pragma unroll
            for (int k = 0; k < T; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    x[k][j] = *(const float4_t*)(a.h + ((size_t)min(s + j, a.slices - 1) * a.M + min(row_of(k), a.M - 1)) * ranks + part * a.R + min(4 * l, a.R - 4));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < T; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (s + j < a.slices) v[k] += x[k][j];
        }
#pragma unroll
        for (int k = 0; k < T; ++k) {
            const bool there = i0 + k < tiles && row_of(k) < a.M;
            who[k] = !there ? -2 : who[k] < 0 || who[k] >= a.n ? -1 : who[k];
            rank[k] = a.ranks ? a.ranks[max(who[k], 0)] : a.R, scale[k] = a.scales ? a.scales[max(who[k], 0)] : 1.f;
        }
#pragma unroll
        for (int k = 0; k < T; ++k) rank[k] = who[k] < 0 ? 0 : min(max(rank[k], 0), a.R);
#pragma unroll
        for (int k = 0; k < T; ++k) {
            if (i0 + k >= tiles) continue;
            const int i = (i0 + k) * kRows + (t >> 4);
            uint32_t top = 0;
            float up = 1.f, down = 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[k][j] = 4 * l + j < rank[k] ? v[k][j] * scale[k] : 0.f;   // ranks past the adapter's are zeros times x, or were not written
                top = max(top, magnitude(v[k][j]));
            }
            if constexpr (!BF16) up = to_range(top, down);
            uint32_t term[2][NT];
#pragma unroll
            for (int j = 0; j < 2; ++j) terms_of<BF16, NT>(v[k][2 * j] * up, v[k][2 * j + 1] * up, term[j]);
            if (4 * l < kStep * RS) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    *(u32x2_t*)(hb + (((i0 + k) * NT + j) * kRows + (t >> 4)) * stride + 4 * l) = u32x2_t{term[0][j], term[1][j]};
            }
            if (l == 0) ids[i] = who[k], back[i] = down;
        }
    }
    __syncthreads();
    if (n >= n1) return;
    u32x4_t w[RS][8];
    int held = -2;
    auto take = [&](int one) {   // the adapter's columns of b: lane (c, g) has ranks 8 g .. of columns 8 c + t
        held = one;
        const int rank = (a.ranks ? (min(max(__builtin_amdgcn_readfirstlane(a.ranks[one]), 0), a.R) + 7) & ~7 : a.R);
        const __amdgpu_buffer_rsrc_t r = make_rsrc(a.b + ((size_t)one * a.N + n) * a.R, (uint32_t)min(kGroup, n1 - n) * 2u * a.R);
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[s][k] = bitcast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(
                    r, kStep * s + 8 * g < rank ? (uint32_t)((8 * c + k) * a.R + kStep * s + 8 * g) * 2u : kNowhere, 0, 0));
    };
#pragma unroll 1
    for (int i0 = 0; i0 < tiles; i0 += D) {
#pragma unroll
        for (int slot = 0; slot < D; ++slot) {
            const int i = i0 + slot;
            const __amdgpu_buffer_rsrc_t ry = of_tile(a.y, i);
            const int mine = i < tiles && lane < kRows ? ids[min(i, tiles - 1) * kRows + lane] : -2;
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = BF16 ? 1.f : back[min(i, tiles - 1) * kRows + 4 * g + k];
            auto put = [&](const float4_t* acc, uint32_t members) {
                u32x4_t out[4][S::kWords];
                S::result(acc, base[slot], f, out);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int e = 0; e < S::kWords; ++e)
                        __builtin_amdgcn_raw_buffer_store_b128(out[k][e], ry, (members >> (4 * g + k)) & 1u ? at[k] : kNowhere, 16 * e, 0);
            };
            float4_t acc[8];
            uint64_t left = __builtin_amdgcn_ballot_w64(mine >= 0);
            for (int nth = 0; left; ++nth) {
                const int one = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
                const uint64_t same = __builtin_amdgcn_ballot_w64(mine == one);
                left &= ~same;
                if (nth % a.turns != turn) continue;
                if (one != held) take(one);
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < RS; ++s) S::multiply(w[s], hb + (size_t)i * NT * kRows * stride, stride, s, acc);
                put(acc, (uint32_t)same);
            }
            const uint64_t none = __builtin_amdgcn_ballot_w64(mine == -1);
            if (none && turn == 0 && a.base != a.y) {   // base copied, the sign of -0 too
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = float4_t{-0.f, -0.f, -0.f, -0.f};
                put(acc, (uint32_t)none);
            }
            load_base(slot, i + D);
        }
    }
}

typedef void (*kernel_t)(LoraArgs);

// The kernels by type and sizes.
template <bool BF16, int Y>
kernel_t both(int R) {
    return R <= 16 ? lora_both_kernel<BF16, 1, Y> : R <= 32 ? lora_both_kernel<BF16, 2, Y> : lora_both_kernel<BF16, 4, Y>;
}
template <bool BF16, int Y>
kernel_t second(int rs) {
    return rs == 1   ? lora_second_kernel<BF16, Y, 1>
           : rs == 2 ? lora_second_kernel<BF16, Y, 2>
           : rs == 4 ? lora_second_kernel<BF16, Y, 4>
                     : lora_second_kernel<BF16, Y, 8>;
}
template <bool BF16, int Y>
kernel_t rows(int rs) {
    return rs == 1 ? lora_rows_kernel<BF16, Y, 1> : lora_rows_kernel<BF16, Y, 2>;
}
template <bool BF16, int MT>
kernel_t first(int rk) {
    return rk == 1   ? lora_first_kernel<BF16, 1, MT>
           : rk == 2 ? lora_first_kernel<BF16, 2, MT>
           : rk == 3 ? lora_first_kernel<BF16, 3, MT>
                     : lora_first_kernel<BF16, 4, MT>;
}
template <bool BF16>
kernel_t both(int R, int y) {
    return y == W4A16_F32 ? both<BF16, W4A16_F32>(R) : y == W4A16_F16 ? both<BF16, W4A16_F16>(R) : both<BF16, W4A16_BF16>(R);
}
template <bool BF16>
kernel_t second(int rs, int y) {
    return y == W4A16_F32 ? second<BF16, W4A16_F32>(rs) : y == W4A16_F16 ? second<BF16, W4A16_F16>(rs) : second<BF16, W4A16_BF16>(rs);
}
template <bool BF16>
kernel_t rows(int rs, int y) {
    return y == W4A16_F32 ? rows<BF16, W4A16_F32>(rs) : y == W4A16_F16 ? rows<BF16, W4A16_F16>(rs) : rows<BF16, W4A16_BF16>(rs);
}
template <bool BF16>
kernel_t first(int rk, int mt) {
    return mt == 1 ? first<BF16, 1>(rk) : first<BF16, 4>(rk);
}

// The kernels' dynamic LDS passes the default limit: said once per process and device.
void allow_lds() {
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices || done[dev].load(std::memory_order_acquire)) return;
    auto allow = [](kernel_t k) { (void)hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicLds); };
    for (int y : {W4A16_F16, W4A16_BF16, W4A16_F32}) {
        for (int R : {16, 32, 64}) allow(both<false>(R, y)), allow(both<true>(R, y));
        for (int rs : {1, 2, 4, 8}) allow(second<false>(rs, y)), allow(second<true>(rs, y));
        for (int rs : {1, 2}) allow(rows<false>(rs, y)), allow(rows<true>(rs, y));
    }
    for (int rk : {1, 2, 3, 4})
        for (int mt : {1, 4}) allow(first<false>(rk, mt)), allow(first<true>(rk, mt));
    done[dev].store(true, std::memory_order_release);
}

struct Plan {
    bool split;           // two launches
    int rk, mt, rs;       // the kernels' template arguments
    int first_threads, threads, turns, first_turns, first_groups, cols, slices;
    int run;              // row tiles of a workgroup of the second launch; 0: not by runs
    long long tiles, first_tiles;
    size_t ws;            // for this many rows and any fewer
};

Plan make_plan(int M, int N, int K, int R, int parts) {
    Plan p{};
    const long long cus = w4h::cu_count(), k_units = (K + kUnit - 1) / kUnit;
    // Tiles of 64 rows in the first product read A less often, tiles of 16 are four times as many workgroups (40 drawn shapes
    // of 257 to 1024 rows, geometric means: 22.9 us with this bound, 23.9 with 256, 22.5 with 1024).
    const bool many = M > 512;
    p.tiles = (M + kRows - 1) / kRows;
    p.rs = R <= 32 ? 1 : R <= 64 ? 2 : R <= 128 ? 4 : 8;
    // One launch where a workgroup's read of all of a part's a costs less than a second launch, for one tile of rows: its LDS
    // fills a CU.  (R K = 80000: one launch 8 to 11 us, two 11; 120000: 11 to 13 and 10 to 14; 235000: 14.2 and 12.1; 600000: 28 and 15.)
    p.split = M > kRows || (long long)R * K > 100000 || p.rs > 2;
    const int rows = p.split ? parts * R : R;            // of a that a workgroup multiplies
    p.rk = rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 48 && p.split ? 3 : 4;
    p.mt = many ? 4 : 1;
    p.threads = p.split ? 256 : 64 * both_waves(p.rk);
    const long long least = 4 * kGroup;                  // columns of a block: a group for each of four waves at least
    p.slices = 1;
    if (p.split && M > 64 && p.rs <= 2) {
        // (64 rows of 48 adapters through gate/up: 45.4 us like this, 32.2 like below; 60 drawn shapes of 65 to 512 rows: 20.8 and 21.7.)
        // By runs of row tiles, the fewest with which all workgroups are on the GPU at once, two per
        // CU; where one-tile runs leave places, several workgroups share a tile's adapters.
        p.cols = (int)least;
        const long long blocks = (N + least - 1) / least + parts - 1, places = 2 * cus / blocks, most = p.rs == 1 ? 16 : 8;
        const long long run = places ? (p.tiles + places - 1) / places : most, share = places / p.tiles, one = M < kRows ? M : kRows;
        p.run = (int)(run < most ? run : most);
        p.turns = (int)(share < 1 ? 1 : share < one ? share : one);
    } else {
        // A workgroup for each adapter that a tile may have (more than 64 rows are as often a few
        // prompts': a quarter of them, the others looped over), and column blocks for two workgroups per CU.
        const int one = M < kRows ? M : M <= 64 ? kRows : kRows / 4;
        const long long units = M <= 64 ? M : p.tiles, want = (2 * cus + units - 1) / units, cols = ((N + want - 1) / want + kGroup - 1) / kGroup * kGroup;
        p.cols = (int)(cols < least ? least : cols);
        const long long share = 2 * cus / (p.tiles * ((N + p.cols - 1) / p.cols));
        p.turns = (int)(!many ? one : share < 1 ? 1 : share < kRows ? share : kRows);
    }
    if (p.split) {
        p.first_threads = p.mt > 1 ? 256 : 512;
        p.first_tiles = (M + kRows * p.mt - 1) / (kRows * p.mt);
        p.first_groups = (rows + 16 * p.rk - 1) / (16 * p.rk);
        const long long first = M <= 64 ? M : many ? p.first_tiles : 2 * p.first_tiles, waves = p.first_threads / 64;
        long long s = cus / (first * p.first_groups);                       // a workgroup fills a CU's LDS
        s = s < k_units / (2 * waves) ? s : k_units / (2 * waves);         // two units for each wave at least
        s = s < 16 ? s : 16;
        p.slices = (int)(s < 1 ? 1 : s);
        // Workgroups for a tile's adapters: as above, more where the slices leave CUs
        // (126 rows of 12 adapters, K 160: 10.0 us with 16, 13.5 with 4).
        const long long spare = cus / (p.first_tiles * p.first_groups * p.slices);
        const int some = many ? 1 : kRows / 4;
        p.first_turns = M < kRows ? M : M <= 64 || spare >= kRows ? kRows : spare > some ? (int)spare : some;
        // More rows take fewer slices: the workspace is for the most rows of partial sums that M rows or fewer
        // have, so that the largest batch's serves every smaller one.  A launch of one workgroup a row, of two
        // for 16 and of one for 64 rows has at most cus workgroups as soon as it has two slices.
        long long most = M;
        auto up_to = [&](long long m, long long rows_of_one, long long units) {
            const long long on_all = rows_of_one * cus / p.first_groups, sliced = (units < 16 ? units : 16) * (m < M ? m : M);
            const long long here = on_all < sliced ? on_all : sliced;
            most = most > here ? most : here;
        };
        up_to(64, 1, k_units / 16);
        if (M > 64) up_to(512, 8, k_units / 16);
        if (many) up_to(M, 64, k_units / 8);
        p.ws = w4h::ws_bytes((size_t)most * parts * R * sizeof(float));
    }
    return p;
}

size_t h_bytes(int rs, int terms) {   // hf, back, hb
    return (kRows * (kStep * rs + 4) + kRows) * sizeof(float) + (size_t)terms * kRows * (kStep * rs + 8) * 2;
}
size_t run_bytes(int run, int rs, int terms) { return (size_t)run * kRows * (8 + (size_t)terms * (kStep * rs + 8) * 2); }   // ids, back, hb

// Workgroups of the launches.
long long first_blocks(const Plan& p) {
    const long long each = p.first_tiles * p.first_groups * p.slices;
    return p.split ? (p.mt > 1 ? (each + 7) / 8 * 8 : each) * p.first_turns : 0;
}
long long second_blocks(const Plan& p, long long blocks) {
    return p.turns * (p.run ? ((p.tiles + p.run - 1) / p.run * blocks + 7) / 8 * 8 : p.tiles * blocks);
}

int check_shape(int M, int N, int K, int R, int parts) {
    if (M < 1 || M > (1 << 26) || N < 8 || N > (1 << 24) || N % 8 || K < 8 || K > (1 << 20) || K % 8 || R < 8 || R > kMaxR || R % 8 ||
        parts < 1 || parts > LORA_MAX_PARTS)
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

// Whether the launches' sizes pass, with the columns' blocks of each part at most one more than its share.
bool fits(const Plan& p, int N, int parts) {
    return second_blocks(p, (N + p.cols - 1) / p.cols + parts) * p.threads <= kMaxLanes && first_blocks(p) * p.first_threads <= kMaxLanes;
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
    if (n_adapters < 1 || ldx < K || ldx % 8 || ldx > (1 << 24) || ldy < N || ldy % 8 || ldy > (1 << 25)) return W4A16_ERR_SHAPE;
    if (parts > 1 && !part_cols) return W4A16_ERR_NULL;
    LoraArgs g{};
    for (int i = 0; i < parts; ++i) {
        const int cols = parts == 1 && !part_cols ? N : part_cols[i];
        if (cols < 8 || cols > N - g.part_start[i] || (i + 1 < parts && cols % 64)) return W4A16_ERR_SHAPE;
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
    g.ldx = ldx, g.ldy = ldy;
    g.n = n_adapters, g.M = M, g.N = N, g.K = K, g.R = R, g.parts = parts;
    g.cols = p.cols, g.turns = p.turns, g.first_turns = p.first_turns, g.slices = p.slices;
    g.first_tiles = (uint32_t)p.first_tiles, g.first_groups = p.first_groups, g.run = p.run;
    for (int i = 0; i < parts; ++i) {
        const int cols = g.part_start[i + 1] - g.part_start[i];
        g.block_start[i + 1] = g.block_start[i] + (cols + p.cols - 1) / p.cols;
    }
    const bool bf16 = dtype == W4A16_BF16;
    const int terms = bf16 && y_dtype == W4A16_F32 ? 3 : 2;
    const hipStream_t st = (hipStream_t)stream;
    const size_t lds = p.run ? run_bytes(p.run, p.rs, terms)
                             : (p.split ? 4 * kSecondStages * (size_t)kStepBytes : first_lds(p.rk, 1, both_waves(p.rk))) + h_bytes(p.rs, terms);
    allow_lds();
    w4h::begin_launches();
    if (p.split) {
        const kernel_t k = bf16 ? first<true>(p.rk, p.mt) : first<false>(p.rk, p.mt);
        hipLaunchKernelGGL(k, dim3((unsigned)first_blocks(p)), dim3(p.first_threads), first_lds(p.rk, p.mt, p.first_threads / 64), st, g);
    }
    const kernel_t k = p.run     ? (bf16 ? rows<true>(p.rs, y_dtype) : rows<false>(p.rs, y_dtype))
                       : p.split ? (bf16 ? second<true>(p.rs, y_dtype) : second<false>(p.rs, y_dtype))
                                 : (bf16 ? both<true>(R, y_dtype) : both<false>(R, y_dtype));
    hipLaunchKernelGGL(k, dim3((unsigned)second_blocks(p, g.block_start[parts])), dim3(p.threads), lds, st, g);
    w4h::note_variant("%s launches=%lld ranks=%lld rows=%lld turns=%lld cols=%lld slices=%lld run=%lld", "lora", p.split ? 2 : 1, 16 * p.rk, 16 * p.mt, p.turns,
                      p.cols, p.slices, p.run);
    return w4h::launch_status();
}
