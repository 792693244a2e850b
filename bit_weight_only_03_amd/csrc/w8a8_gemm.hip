// w8a8_gemm.hip -- y = x . w^T for e4m3 operands with one fp32 scale per row
// and 128 k of x and one per 128 x 128 block of w.
//
// Both operands come in rows of K bytes, and v_mfma_f32_16x16x128_f8f6f4 takes
// exactly one scale block (128 k) of 16 rows of each: the block's sum leaves
// the matrix unit in fp32 and takes its scales' product in one fp32 fma per
// output.  w is the A operand and x the B operand, so a lane's four results
// share one row m of x, hence one scale, and are four consecutive columns n
// of y.
//
// Rows go to LDS by direct loads (buffer_load ... lds), 128 bytes of 8 rows
// per instruction: whole cache lines, where the operand layout itself (16 rows
// by 16 bytes for each quarter wave) would touch half lines.  A row's eight 16-byte
// chunks are permuted by a key of the row on the way, so that the operand
// reads (16 bytes at one chunk of 16 rows) are free of bank conflicts.
//
// Lane l of an operand holds row l & 15 and the chunks l >> 4 and 4 + (l >> 4)
// of its 128 bytes.  Which k an MFMA slot stands for does not matter as long as
// both operands agree.
//
// Roundings: the matrix unit aligns the products of 8 consecutive k to their
// largest and drops what lies below 2^-13 of it (measured: rms 2e-6 of
// sum |x w|); everything from the block's sum on is fp32, rounded once to y's
// type.
#include <math.h>

#include <atomic>

#include "w8a8_common.h"

using namespace w4k;

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kOutside = 0x80000000u;   // an offset past every descriptor here: reads zeros
constexpr int kStepK = 128;                  // k per step: one scale block, one MFMA
constexpr int kMaxSplit = 64;
constexpr int kMaxDynamicLds = 160 * 1024;
constexpr int kMaxDevices = 64;
constexpr int kMaxM = 1 << 26;               // a block's x_scales in one 32-bit descriptor

struct GemmArgs {
    const uint8_t* x;
    const float* x_scales;
    const uint8_t* w;
    const float* w_scales;
    void* y;
    float* part;          // fp32 partial sums of K slices
    unsigned* counters;   // one per output tile, zero between calls
    int y_dtype;
    int M, N, K;
    int kb;               // scale blocks of K
    int S;                // K slices
    int tiles_n, tiles_m;
};

__device__ __forceinline__ float4_t mfma_block(const i32x8_t& a, const i32x8_t& b) {
    // Formats 0, 0: both e4m3.  Scale operands of constant 0 select the form without scales.
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, float4_t{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                            0, 0, 0, 0);
}

// The operand whose row starts at p in LDS, chunks permuted with key.
__device__ __forceinline__ i32x8_t operand(const uint8_t* p, int chunk, int key) {
    const i32x4_t lo = *(const i32x4_t*)(p + 16 * (chunk ^ key));
    const i32x4_t hi = *(const i32x4_t*)(p + 16 * ((chunk + 4) ^ key));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)to, 16, voff, soff, 0, 0);
}

// Four consecutive n of one row of y.  n and N are multiples of 4 and 8: a
// quad is whole or absent.
__device__ __forceinline__ void store4(const GemmArgs& a, int m, int n, const float* f) {
    if (m >= a.M || n >= a.N) return;
    const size_t o = (size_t)m * a.N + n;
    if (a.y_dtype == W4A16_F32)
        *(float4_t*)((float*)a.y + o) = float4_t{f[0], f[1], f[2], f[3]};
    else if (a.y_dtype == W4A16_F16)
        *(u32x2_t*)((uint16_t*)a.y + o) = u32x2_t{pk_f16(f[0], f[1]), pk_f16(f[2], f[3])};
    else
        *(u32x2_t*)((uint16_t*)a.y + o) = u32x2_t{pk_bf16(f[0], f[1]), pk_bf16(f[2], f[3])};
}

// The merge of K slices inside the launch.  Of every slice's workgroup the
// first `threads` threads hold C partial sums each.  They store them
// (coherently across the device, thread-contiguous); the workgroup
// counts itself in, and the last to arrive adds all slices in slice order: the
// result does not depend on who was last.  True for that workgroup, whose f
// then holds the sums.  No workgroup waits for another.
template <int C>
__device__ __forceinline__ bool merge_slices(const GemmArgs& a, int tile, int slice, int threads, bool live,
                                             unsigned* arrived, float* f) {
    const int t = threadIdx.x;
    float* const base = a.part + (size_t)tile * a.S * C * threads;
    if (live) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            __hip_atomic_store(base + ((size_t)slice * C + c) * threads + t, f[c], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    __builtin_amdgcn_s_waitcnt(0);   // this thread's stores are done
    __syncthreads();
    if (t == 0) *arrived = __hip_atomic_fetch_add(a.counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (*arrived != (unsigned)(a.S - 1)) return false;
    if (t == 0) __hip_atomic_store(a.counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (live) {
        float v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = 0.f;
        for (int s = 0; s < a.S; ++s)
#pragma unroll
            for (int c = 0; c < C; ++c)
                v[c] += __hip_atomic_load(base + ((size_t)s * C + c) * threads + t, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int c = 0; c < C; ++c) f[c] = v[c];
    }
    return true;
}

// ---- few rows ----
//
// Bound by one read of w.  A workgroup takes NT tiles of 16 columns and one
// slice of K; its W waves take the slice's 128-k units in turn, each through
// a private ring of RD slots in LDS ([16 NT rows of w][XR rows of x] x 128
// bytes) that it fills RD units ahead and waits on alone: no barrier until the
// waves' sums are added at the end.  MT tiles of 16 rows of x (XR = 8: half a
// tile, whose other half repeats it and is not stored).
//
// Four waves per workgroup and two workgroups per CU keep about 100 KB of w on
// its way to each CU.  1 x 34816 x 5120 takes 32 us (5.6 TB/s of w), 32 rows of it
// 42, 1 x 7168 x 5120 9 us (4 TB/s: about 5 us are a launch's start, its first
// loads and its last sum).  K slices pay only where tiles leave most CUs idle:
// 64 x 7168 x 5120 takes 16.6 us whole, 22 and 30 in two and four slices.
// Starting each tile at another k (other memory channels at one time) changed nothing.
constexpr int kTableFloats = 2048;   // products of scales a workgroup holds

template <int MT, int XR, int NT, int RD, int W>
__global__ __launch_bounds__(W * 64, 2) void w8a8_skinny_kernel(GemmArgs a) {
    constexpr int kSlot = (16 * NT + XR) * kStepK;
    constexpr int kLoads = 2 * NT + XR / 8;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    float* const table = (float*)(smem + W * RD * kSlot);   // [unit of the slice][XR]
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63;

    // Consecutive workgroups go to the XCDs in turn; the row blocks of one
    // tile and slice sit 8 apart, on one XCD, whose L2 then serves w again.
    const int r = blockIdx.x >> 3, mb = r % a.tiles_m, id = (r / a.tiles_m) * 8 + (blockIdx.x & 7);
    if (id >= a.tiles_n * a.S) return;
    const int tile = id / a.S, slice = id % a.S;
    const int n0 = tile * 16 * NT, m0 = mb * XR;
    const int b0 = (int)((long long)a.kb * slice / a.S), b1 = (int)((long long)a.kb * (slice + 1) / a.S);
    const int units = b1 - b0, nu = units > wave ? (units - wave + W - 1) / W : 0;

    // The products of scales of this slice, once: x_scales[b][m] w_scales[n/128][b].
    constexpr int kPer = (kTableFloats + W * 64 - 1) / (W * 64);
    float sx[kPer], sw[kPer];
    const float* const ws = a.w_scales + (size_t)(n0 >> 7) * a.kb;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = i * W * 64 + t, u = e / XR, m = m0 + e % XR;
        sx[i] = sw[i] = 0.f;
        if (u < units && m < a.M) {
            sx[i] = a.x_scales[(size_t)(b0 + u) * a.M + m];
            sw[i] = ws[b0 + u];
        }
    }
    __builtin_amdgcn_sched_barrier(0);

    const int rows_n = min(16 * NT, a.N - n0), rows_m = min(XR, a.M - m0);
    const uint32_t K = a.K;
    const uint8_t* const wp = a.w + (size_t)n0 * K;
    const uint8_t* const xp = a.x + (size_t)m0 * K;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(wp, rows_n * K), rx = make_rsrc(xp, rows_m * K);
    const __amdgpu_buffer_rsrc_t none = make_rsrc(wp, 0);   // a unit that does not exist reads zeros
    uint8_t* const ring = smem + wave * RD * kSlot;
    const int row8 = lane >> 3, chunk = (lane & 7) ^ row8;   // slot chunk lane & 7 of row row8 holds this one
    const uint32_t lane_off = row8 * K + 16u * chunk;
    const int last = a.kb - 1, tail = (int)K - last * kStepK;   // bytes of the last unit's rows
    const uint32_t tail_off = 16 * chunk < tail ? lane_off : kOutside;

    auto issue = [&](int i) {
        const int u = b0 + wave + i * W;
        const bool there = i < nu;
        const uint32_t off = u == last ? tail_off : lane_off;
        const uint32_t k = (uint32_t)u * kStepK;
        uint8_t* const slot = ring + (i % RD) * kSlot;
#pragma unroll
        for (int j = 0; j < 2 * NT; ++j) {
            uint32_t o = off + 8u * j * K;
            o = off == kOutside ? kOutside : o;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(there ? rw : none, (lds_ptr_t)(slot + j * 1024), 16, o, k, 0, kAuxNT);
        }
#pragma unroll
        for (int j = 0; j < XR / 8; ++j) {
            uint32_t o = off + 8u * j * K;
            o = off == kOutside ? kOutside : o;
            load_lds(there ? rx : none, slot + 16 * NT * kStepK + j * 1024, o, k);
        }
    };
#pragma unroll
    for (int i = 0; i < RD; ++i) issue(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = i * W * 64 + t;
        if (e < units * XR) table[e] = sx[i] * sw[i];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    float4_t acc[NT][MT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = float4_t{0.f, 0.f, 0.f, 0.f};
    const int c = lane & 15, g = lane >> 4, key = c & 7;
    for (int i = 0; i < nu; ++i) {
        // All but the RD - 1 younger units' loads have arrived.
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((RD - 1) * kLoads) : "memory");
        const uint8_t* const slot = ring + (i % RD) * kSlot;
        i32x8_t wf[NT], xf[MT];
        float s[MT];
#pragma unroll
        for (int n = 0; n < NT; ++n) wf[n] = operand(slot + (16 * n + c) * kStepK, g, key);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int row = XR == 8 ? c & 7 : 16 * m + c;
            xf[m] = operand(slot + (16 * NT + row) * kStepK, g, key);
            s[m] = table[(wave + i * W) * XR + row];
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read: it may be filled again
        issue(i + RD);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float4_t d = mfma_block(wf[n], xf[m]);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[n][m][q] = __builtin_fmaf(d[q], s[m], acc[n][m][q]);
            }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // no load may still be on its way into LDS
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    // The waves' sums, added in wave order: [wave][tile][4][lane].
    float* const red = (float*)smem;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) red[((wave * NT * MT + n * MT + m) * 4 + q) * 64 + lane] = acc[n][m][q];
    __syncthreads();
    constexpr int kTiles = NT * MT;
    static_assert(kTiles <= W, "one operand tile per wave");
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    const int m = m0 + 16 * (wave % MT) + c, n = n0 + 16 * (wave / MT) + 4 * g;
    const bool live = wave < kTiles && m < a.M && (XR != 8 || c < 8);
    if (live) {
#pragma unroll
        for (int wv = 0; wv < W; ++wv)
#pragma unroll
            for (int q = 0; q < 4; ++q) f[q] += red[((wv * kTiles + wave) * 4 + q) * 64 + lane];
    }
    if (a.S > 1 && !merge_slices<4>(a, tile * a.tiles_m + mb, slice, kTiles * 64, live, (unsigned*)table, f)) return;
    if (live) store4(a, m, n, f);
}

// ---- many rows ----
//
// Bound by the matrix units.  A workgroup of WGM x WGN waves takes BM rows of x
// by BN rows of w; each step's 128 k go to LDS rings, x's of XD blocks and w's of
// three, while an older block is multiplied: one barrier per step.
//
// 8192 x 8192 x 8192 takes 454 us (2.42 PFLOP/s; the library's product with one
// scale for all of x and w reaches 2.6), 4096 x 34816 x 5120 650 to 680 (2.14 to
// 2.24: its 2176 tiles are 8.5 rounds of 256 CUs).  A step of the largest tile is
// 32 MFMAs of 32 clocks for each of a SIMD's two waves, and beside them 24 LDS
// reads and 128 fmas per wave; these run under products only if a wave never
// waits for the product it has just asked for: hence kLag.  At 64 to 128 rows
// w's stream bounds it (128 x 34816 x 5120: 59 us, 3 TB/s of w); tiles of 64 x 64
// and 128 x 64 and deeper rings of x were within 5 percent there.
//
// Inside a wave's WN columns, row r of operand tile t is column
// (r >> 2) WN/4 + 4 t + (r & 3): a lane's results over all tiles are then WN/4
// consecutive columns of one row of y, stored 16 bytes at a time.  The key of
// such a row follows r & 7, as its 8 neighbouring lanes need.
template <int BM, int BN, int WGM, int WGN, int XD>
__global__ __launch_bounds__(WGM * WGN * 64, 2) void w8a8_tiled_kernel(GemmArgs a) {
    constexpr int W = WGM * WGN, WM = BM / WGM, WN = BN / WGN, MT = WM / 16, NT = WN / 16;
    constexpr int kXBuf = BM * kStepK, kWBuf = BN * kStepK;
    constexpr int XL = BM / (8 * W), WL = BN / (8 * W);   // loads per wave and step
    constexpr int kAll = XL + WL;
    constexpr int kLag = 3;   // products under way between one and its scaling (4096 x 34816 x 5120 with 1: 691, 2: 678, 3: 665, 4: 672 us)
    static_assert(XL >= 1 && WL >= 1 && WN <= 128 && WN >= 32, "tile shape");
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63;
    const int wm = wave % WGM, wn = wave / WGM;

    // Tiles go to the XCDs in contiguous shares, each walked in columns of
    // kGroup row tiles, so that an XCD's workgroups share rows of both operands in its L2.
    constexpr int kGroup = 8;
    const int total = a.tiles_m * a.tiles_n * a.S;
    const int share = (total + 7) / 8;
    const int id = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= share || id >= total) return;
    const int slice = id % a.S, at = id / a.S;
    const int band = at / (kGroup * a.tiles_n), in_band = at % (kGroup * a.tiles_n);
    const int band_m = min(kGroup, a.tiles_m - band * kGroup);
    const int tm = band * kGroup + in_band % band_m, tn = in_band / band_m;
    const int m0 = tm * BM, n0 = tn * BN;
    const int b0 = (int)((long long)a.kb * slice / a.S), b1 = (int)((long long)a.kb * (slice + 1) / a.S);

    const uint32_t K = a.K;
    const int rows_n = min(BN, a.N - n0), rows_m = min(BM, a.M - m0);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)n0 * K, rows_n * K);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)m0 * K, rows_m * K);
    const int last = a.kb - 1, tail = (int)K - last * kStepK;
    // Load j of a wave: rows 8 (j W + wave) + lane / 8.
    const int row8 = lane >> 3;
    const int wkey = (row8 & 3) | ((((8 * wave) / (WN / 4)) & 1) << 2);
    static_assert((8 * W / (WN / 4)) % 2 == 0, "a wave's rows of w keep one key");
    const int xchunk = (lane & 7) ^ row8, wchunk = (lane & 7) ^ wkey;
    uint32_t xoff[XL], woff[WL];
#pragma unroll
    for (int j = 0; j < XL; ++j) xoff[j] = (uint32_t)(8 * (j * W + wave) + row8) * K + 16u * xchunk;
#pragma unroll
    for (int j = 0; j < WL; ++j) woff[j] = (uint32_t)(8 * (j * W + wave) + row8) * K + 16u * wchunk;

    // Load j of this wave: of block b of x into ring slot i (of XD), of w into slot i (of 3).
    auto issue_x = [&](int j, int b, int i) {
        load_lds(rx, smem + i * kXBuf + (j * W + wave) * 1024, b == last && 16 * xchunk >= tail ? kOutside : xoff[j],
                 (uint32_t)b * kStepK);
    };
    auto issue_w = [&](int j, int b, int i) {
        load_lds(rw, smem + XD * kXBuf + i * kWBuf + (j * W + wave) * 1024,
                 b == last && 16 * wchunk >= tail ? kOutside : woff[j], (uint32_t)b * kStepK);
    };

    const int c = lane & 15, g = lane >> 4, key = c & 7;
    const int nw = n0 + wn * WN;   // this wave's first column; all of them in one scale block
    const float* const ws = a.w_scales + (size_t)(min(nw, a.N - 1) >> 7) * a.kb;
    const uint32_t xs_off = (uint32_t)(m0 + wm * WM + c) * 4u;   // rows past M read scales of 0
    float4_t acc[NT][MT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = float4_t{0.f, 0.f, 0.f, 0.f};

    float sx[MT], sw;
    const __amdgpu_buffer_rsrc_t rws = make_rsrc(ws, (uint32_t)a.kb * 4u);
    auto scales = [&](int b) {
        const __amdgpu_buffer_rsrc_t rxs = make_rsrc(a.x_scales + (size_t)b * a.M, (uint32_t)a.M * 4u);
        sw = bitcast<float>(__builtin_amdgcn_raw_buffer_load_b32(rws, 0, (uint32_t)b * 4u, 0));
#pragma unroll
        for (int m = 0; m < MT; ++m)
            sx[m] = bitcast<float>(__builtin_amdgcn_raw_buffer_load_b32(rxs, xs_off + 64u * m, 0, 0));
    };
    // Loads are waited for by their number, in the order of the steps: x and w
    // of a block, then (XD = 3) the next block's scales, x and w, or (XD = 2) the next w.
    const int second = min(b0 + 1, b1 - 1);
    if constexpr (XD == 2) scales(b0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < XL; ++j) issue_x(j, b0, 0);
#pragma unroll
    for (int j = 0; j < WL; ++j) issue_w(j, b0, 0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (XD == 3) {
        scales(b0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < XL; ++j) issue_x(j, second, 1);
    }
#pragma unroll
    for (int j = 0; j < WL; ++j) issue_w(j, second, 1);
    __builtin_amdgcn_sched_barrier(0);
    float s[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) s[m] = sx[m] * sw;
    const uint8_t* const xl = smem + (wm * WM + c) * kStepK;
    const uint8_t* const wl = smem + XD * kXBuf + (wn * WN + (c >> 2) * (WN / 4) + (c & 3)) * kStepK;
    int xs = 0, ws3 = 0;
    constexpr int kYounger = XD == 2 ? WL : XL + WL + MT + 1;   // loads issued after this block's last
    for (int b = b0; b < b1; ++b) {
        // This wave's loads of this block have arrived (younger ones may still
        // be on their way) and its reads of the last block are done; after the
        // barrier that holds for every wave.
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kYounger) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const uint8_t* const xb = xl + xs * kXBuf;
        const uint8_t* const wb = wl + ws3 * kWBuf;
        // The slots read in the last step take the loads of this one.
        const int xfill = xs == 0 ? XD - 1 : xs - 1, wfill = ws3 == 0 ? 2 : ws3 - 1;
        xs = xs == XD - 1 ? 0 : xs + 1;
        ws3 = ws3 == 2 ? 0 : ws3 + 1;
        i32x8_t xf[MT], wf[2];
        wf[0] = operand(wb, g, key);
#pragma unroll
        for (int m = 0; m < MT; ++m) xf[m] = operand(xb + 16 * m * kStepK, g, key);
        // The next step's loads; the last step repeats its own, which nothing reads.
        const int next = min(b + 1, b1 - 1), next2 = min(b + 2, b1 - 1), nextx = XD == 3 ? next2 : next;
        scales(next);
        __builtin_amdgcn_sched_barrier(0);
        // The block sums of kLag products are under way while an older one is scaled and added.
        float4_t d[kLag + 1];
#pragma unroll
        for (int j = 0; j < NT * MT + kLag; ++j) {
            const int n = j / MT, m = j % MT;
            if (j < NT * MT) {
                if (m == 0) {
                    if (n + 1 < NT) wf[(n + 1) & 1] = operand(wb + 4 * (n + 1) * kStepK, g, key);
                    // The next loads, over the first three quarters of the step.
                    const int lo = min(kAll, (n * kAll * 4 + 3 * NT - 1) / (3 * NT));
                    const int hi = min(kAll, ((n + 1) * kAll * 4 + 3 * NT - 1) / (3 * NT));
#pragma unroll
                    for (int i = 0; i < kAll; ++i) {
                        if (i < lo || i >= hi) continue;
                        if (i < XL) issue_x(i, nextx, xfill);
                        else issue_w(i - XL, next2, wfill);
                    }
                }
                d[j % (kLag + 1)] = mfma_block(wf[n & 1], xf[m]);
            }
            if (j >= kLag) {
                const int jj = j - kLag, nn = jj / MT, mm = jj % MT;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[nn][mm][q] = __builtin_fmaf(d[jj % (kLag + 1)][q], s[mm], acc[nn][mm][q]);
            }
            __builtin_amdgcn_sched_barrier(0);   // products and sums stay in this order
        }
        // The next step's scales, from loads older than its operands'.
#pragma unroll
        for (int m = 0; m < MT; ++m) s[m] = sx[m] * sw;
    }
    // The last loads, which nothing reads, are done before LDS is reused or released.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (a.S > 1) {
        if (!merge_slices<NT * MT * 4>(a, tm * a.tiles_n + tn, slice, W * 64, true, (unsigned*)smem, (float*)acc)) return;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = m0 + wm * WM + 16 * m + c, col = nw + g * (WN / 4);
        if (row >= a.M) continue;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {   // 8 columns, whole or absent
            if (col + 4 * n >= a.N) continue;
            const float f[8] = {acc[n][m][0],     acc[n][m][1],     acc[n][m][2],     acc[n][m][3],
                                acc[n + 1][m][0], acc[n + 1][m][1], acc[n + 1][m][2], acc[n + 1][m][3]};
            store8(a.y, a.y_dtype, (size_t)row * a.N + col + 4 * n, f);
        }
    }
}

// ---- plan ----

typedef void (*kernel_t)(GemmArgs);

struct Plan {
    kernel_t kernel;
    const char* name;
    int bm, bn;        // rows and columns of a tile
    int threads;
    size_t lds;
    int S;
    int floats;        // partial sums of a tile and slice
    long long tiles_m, tiles_n;
    long long blocks;
    size_t ws;
};

template <int MT, int XR, int NT, int RD, int W>
Plan skinny_plan(const char* name) {
    Plan p{};
    p.kernel = w8a8_skinny_kernel<MT, XR, NT, RD, W>;
    p.name = name;
    p.bm = XR, p.bn = 16 * NT, p.threads = W * 64;
    p.lds = (size_t)W * RD * (16 * NT + XR) * kStepK + kTableFloats * sizeof(float);
    p.floats = 16 * MT * 16 * NT;
    return p;
}

template <int BM, int BN, int WGM, int WGN, int XD>
Plan tiled_plan(const char* name) {
    Plan p{};
    p.kernel = w8a8_tiled_kernel<BM, BN, WGM, WGN, XD>;
    p.name = name;
    p.bm = BM, p.bn = BN, p.threads = WGM * WGN * 64;
    p.lds = (size_t)(XD * BM + 3 * BN) * kStepK;
    p.floats = BM * BN;
    return p;
}

constexpr size_t kMaxPartials = (size_t)64 << 20;
constexpr int kCounters = (int)(w4h::kWsHead / sizeof(unsigned));

// The kernels, each with what a step takes in microseconds (128 k of a tile; a
// unit for each of the four waves), alone on its CU and beside a second workgroup, what a
// launch takes besides, and the rate at which it streams w from HBM (bytes per
// microsecond: a tile's rows are read 128 bytes at a time, the skinny
// kernels' 512).  Measured on MI355X, K = 5120 and 17408, N = 1024 .. 34816.
// Kernels for far fewer or more rows than M are not looked at (from, to).  The
// skinny ones pay beyond their own rows where there are few columns: 517 x 112
// x 5984 9.0 us against 12.9 with the best tiled one, 100 x 1024 x 5120 7.3 against
// 12.0; with many columns the tiled ones do: 128 x 34816 x 5120 59 against 113.
struct Kernel {
    Plan p;   // all but the counts of tiles, slices and bytes
    int from, to;
    bool skinny;
    float alone, beside, start, stream;
};
const Kernel kKernels[] = {
    {skinny_plan<1, 8, 1, 4, 4>("skinny8x16"), 1, 8, true, 0.27f, 0.45f, 4.0f, 7.0e6f},
    {skinny_plan<1, 8, 2, 3, 4>("skinny8x32"), 1, 8, true, 0.42f, 0.60f, 4.5f, 7.0e6f},
    {skinny_plan<1, 16, 2, 3, 4>("skinny16x32"), 9, 512, true, 0.58f, 0.75f, 4.5f, 7.0e6f},
    {skinny_plan<2, 32, 2, 2, 4>("skinny32x32"), 17, 2048, true, 0.78f, 1.10f, 4.5f, 7.0e6f},
    {tiled_plan<64, 128, 2, 2, 2>("tiled64x128"), 17, 1 << 26, false, 0.53f, 0.79f, 6.0f, 3.3e6f},
    {tiled_plan<128, 128, 2, 2, 2>("tiled128x128"), 65, 1 << 26, false, 0.78f, 1.15f, 6.0f, 3.3e6f},
    {tiled_plan<128, 256, 2, 4, 3>("tiled128x256"), 65, 1 << 26, false, 0.97f, 0.97f, 7.0f, 3.7e6f},
    {tiled_plan<256, 256, 4, 2, 2>("tiled256x256"), 257, 1 << 26, false, 1.60f, 1.60f, 8.0f, 3.3e6f},
};
constexpr int kKernelCount = sizeof kKernels / sizeof kKernels[0];

// The kernel and the slices of K with the least estimated time: rounds of
// workgroups over the CUs, each a start and its steps, not faster than w
// arrives; slices add their partial sums' traffic and the merge.  Slices looked
// at: 1, 2, 4 and 8, and beyond 8 those that fill the CUs halfway, once and to
// their occupancy.  (Between, 3 are faster at some sizes: 512 x 5120 x 17408 71 us
// against 81 with 2.)
//
// The kernels of few rows have to slice a sum whose scales pass their table
// (K > 32768 up to 8 rows, 16384 up to 16): over very many columns those slices
// pass the counters or the partial sums' limit.  Where the kernels meant for M leave
// no plan like this, all are looked at: the tiled ones hold no table.  None is left
// only past a launch's size (M N from about 2^39) or under overridden slices.
Plan make_plan(int M, int N, int K) {
    const int kb = (K + kStepK - 1) / kStepK, cus = w4h::cu_count();
    const int only = w4h::overrides().w8_variant, slices = w4h::overrides().w8_split;
    const bool any = only < 0 || only >= kKernelCount;
    Plan best{};
    float least = 0;
    auto look_at = [&](const Kernel& k) {
        Plan p = k.p;
        p.tiles_m = ((long long)M + p.bm - 1) / p.bm;
        p.tiles_n = ((long long)N + p.bn - 1) / p.bn;   // N + bn - 1 may pass 32 bits
        const long long all = p.tiles_m * p.tiles_n;
        const int tiles = all < (1 << 24) ? (int)all : 1 << 24;   // more never has slices
        const int waves = k.skinny ? p.threads / 64 : 1;          // units a step takes
        const int slots = 2 * p.lds <= (size_t)kMaxDynamicLds ? 2 * cus : cus;
        // The products of scales of a skinny kernel's slice fit its table.
        const int least_S = k.skinny ? (kb * p.bm + kTableFloats - 1) / kTableFloats : 1;
        int last = 0;
        for (int S : {1, 2, 4, 8, cus / tiles / 2, cus / tiles, slots / tiles}) {
            S = slices > 0 ? slices : S;
            S = S < kb / (2 * waves) ? S : kb / (2 * waves);   // two steps at least
            S = S < least_S ? least_S : S;
            S = S < 1 ? 1 : S > kMaxSplit ? kMaxSplit : S;
            if (S <= last) continue;
            last = S;
            if (k.skinny && ((kb + S - 1) / S) * p.bm > kTableFloats) continue;
            const size_t partials = S > 1 ? (size_t)tiles * S * p.floats * sizeof(float) : 0;
            if (S > 1 && (tiles > kCounters || partials > kMaxPartials)) continue;
            p.blocks = k.skinny ? (p.tiles_n * S + 7) / 8 * 8 * p.tiles_m : (all * S + 7) / 8 * 8;
            if (p.blocks * p.threads > kMaxLanes) continue;
            const float wgs = (float)all * S, steps = (float)((kb + S * waves - 1) / (S * waves));
            float t = ceilf(wgs / slots) * (k.start + steps * (wgs > cus ? k.beside : k.alone));
            t = fmaxf(t, k.start + (float)N * K / k.stream);
            if (S > 1) t += 2.0f + 0.3f * S + partials / 2e6f;
            if (best.S == 0 || t < least) {
                least = t;
                best = p;
                best.S = S;
                best.ws = w4h::ws_bytes(partials);
            }
        }
    };
    for (int v = 0; v < kKernelCount; ++v)
        if (any ? M >= kKernels[v].from && M <= kKernels[v].to : v == only) look_at(kKernels[v]);
    if (any && !best.kernel)
        for (const Kernel& k : kKernels) look_at(k);
    return best;
}

// The kernels' dynamic LDS may pass the default limit: said once per process and device.
void allow_lds() {
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices || done[dev].load(std::memory_order_acquire))
        return;
    for (const Kernel& k : kKernels)
        (void)hipFuncSetAttribute((const void*)k.p.kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicLds);
    done[dev].store(true, std::memory_order_release);
}

int check_shape(int M, int N, int K) {
    if (M < 1 || M > kMaxM || N < 8 || N % 8 || K < 16 || K % 16 || K > (1 << 20)) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

}  // namespace

extern "C" int w8a8_workspace_bytes(int M, int N, int K, size_t* bytes) {
    if (!bytes) return W4A16_ERR_NULL;
    if (int rc = check_shape(M, N, K)) return rc;
    const Plan p = make_plan(M, N, K);
    if (!p.kernel) return W4A16_ERR_UNSUPPORTED;
    *bytes = p.ws;
    return W4A16_OK;
}

extern "C" int w8a8_gemm(const void* x, const float* x_scales, const void* w, const float* w_scales,
                         void* y, int y_dtype, int M, int N, int K, void* workspace,
                         size_t workspace_bytes, w4a16_stream_t stream) {
    if (!x || !x_scales || !w || !w_scales || !y) return W4A16_ERR_NULL;
    if (y_dtype != W4A16_F16 && y_dtype != W4A16_BF16 && y_dtype != W4A16_F32) return W4A16_ERR_DTYPE;
    if (int rc = check_shape(M, N, K)) return rc;
    if (!w4h::aligned16(x) || !w4h::aligned16(x_scales) || !w4h::aligned16(w) ||
        !w4h::aligned16(w_scales) || !w4h::aligned16(y) || !w4h::aligned16(workspace))
        return W4A16_ERR_ALIGN;
    const Plan p = make_plan(M, N, K);
    if (!p.kernel) return W4A16_ERR_UNSUPPORTED;
    if (p.ws && !workspace) return W4A16_ERR_NULL;
    if (workspace_bytes < p.ws) return W4A16_ERR_WORKSPACE;
    GemmArgs a{(const uint8_t*)x, x_scales, (const uint8_t*)w, w_scales, y,
               (float*)w4h::ws_part(workspace), (unsigned*)workspace, y_dtype, M, N, K,
               (K + kStepK - 1) / kStepK, p.S, (int)p.tiles_n, (int)p.tiles_m};
    allow_lds();
    w4h::begin_launches();
    hipLaunchKernelGGL(p.kernel, dim3((unsigned)p.blocks), dim3(p.threads), p.lds, (hipStream_t)stream, a);
    w4h::note_variant("w8a8_gemm %s tiles=%lldx%lld slices=%lld threads=%lld lds=%lld", p.name, p.tiles_m, p.tiles_n, p.S,
                      p.threads, p.lds);
    return w4h::launch_status();
}
