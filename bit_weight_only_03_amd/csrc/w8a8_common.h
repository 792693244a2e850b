// w8a8_common.h -- device helpers of the 8-bit block-scaled layer: typed loads
// and stores of 8 consecutive elements, and the e4m3 block scale.
#pragma once

#include "common.h"

namespace w4k {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kScaleBlock = 128;             // columns that share a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 0x1p-60f;      // least magnitude a scale is made for

// Eight consecutive elements at o (8 * element size aligned) as fp32.
__device__ __forceinline__ void load8(const void* p, int dtype, size_t o, float* f) {
    if (dtype == W4A16_F32) {
        const float4_t a = *(const float4_t*)((const float*)p + o);
        const float4_t b = *(const float4_t*)((const float*)p + o + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = a[e], f[4 + e] = b[e];
        return;
    }
    const u32x4_t v = *(const u32x4_t*)((const uint16_t*)p + o);
    if (dtype == W4A16_F16) {
        const half8_t hv = bitcast<half8_t>(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)hv[e];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = bitcast<float>(v[j] << 16);
            f[2 * j + 1] = bitcast<float>(v[j] & 0xffff0000u);
        }
    }
}

// fp32 to two bf16, rounded to nearest even (NaN stays NaN): v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return bitcast<uint32_t>(v);
}
__device__ __forceinline__ uint32_t pk_f16(float a, float b) {
    return as_u(half2_t{(_Float16)a, (_Float16)b});
}

// A store that need not stay in the caches (NT), or an ordinary one.
template <bool NT, typename V>
__device__ __forceinline__ void store(V* p, const V& v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// Eight fp32 values stored in the dtype (16-bit types rounded to nearest even).
template <bool NT = false>
__device__ __forceinline__ void store8(void* p, int dtype, size_t o, const float* f) {
    if (dtype == W4A16_F32) {
        store<NT>((float4_t*)((float*)p + o), float4_t{f[0], f[1], f[2], f[3]});
        store<NT>((float4_t*)((float*)p + o + 4), float4_t{f[4], f[5], f[6], f[7]});
        return;
    }
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = dtype == W4A16_F16 ? pk_f16(f[2 * j], f[2 * j + 1]) : pk_bf16(f[2 * j], f[2 * j + 1]);
    store<NT>((u32x4_t*)((uint16_t*)p + o), v);
}

// v of another lane of the same 16 (a DPP row), by DPP control word.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// The scale of the block that the 16 lanes of a DPP row hold, in all of them.
// Magnitudes are compared as integers: the bit patterns of |n| order as the
// values do, infinity above every finite one and NaN above infinity, so a NaN
// anywhere in the block makes the scale NaN (a float maximum would drop it).
__device__ __forceinline__ float block_scale(const float* n) {
    uint32_t m = bitcast<uint32_t>(kScaleFloor);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, bitcast<uint32_t>(n[e]) & 0x7fffffffu);
    m = max(m, dpp<0xB1>(m));    // lanes 1 apart (quad_perm 1,0,3,2)
    m = max(m, dpp<0x4E>(m));    // lanes 2 apart (quad_perm 2,3,0,1)
    m = max(m, dpp<0x141>(m));   // the quad beside it (row_half_mirror)
    m = max(m, dpp<0x140>(m));   // the other eight lanes (row_mirror)
    return bitcast<float>(m) * (1.0f / kE4m3Max);
}

// Eight values over the scale as e4m3, rounded to nearest even.  |n| / s is at
// most 448 but for the rounding of the quotient, which stays below 464, where
// e4m3 still rounds to 448.
template <bool NT>
__device__ __forceinline__ void store_q8(uint8_t* p, const float* n, float s) {
    const float r = __builtin_amdgcn_rcpf(s);
    u32x2_t v;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(n[4 * j] * r, n[4 * j + 1] * r, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(n[4 * j + 2] * r, n[4 * j + 3] * r, w, true);
        v[j] = (uint32_t)w;
    }
    store<NT>((u32x2_t*)p, v);
}

}  // namespace w4k

constexpr long long kMaxLanes = 0xffffffffLL;   // work-items of a launch
