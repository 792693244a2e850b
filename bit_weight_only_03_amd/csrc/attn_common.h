// attn_common.h -- device helpers of the attentions over a paged cache: waits,
// 16-bit products, the largest and the sum over the lanes of a row, masks.
#pragma once

#include <math.h>

#include <atomic>
#include <type_traits>

#include "w8a8_common.h"

namespace w4k {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef const __attribute__((address_space(1))) void* global_ptr_t;

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kLn2 = 0x1.62e43p-1f;
constexpr int kMaxDevices = 64;
constexpr int kMaxDynamicLds = 160 * 1024;

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

// 2^(m - top), 0 for a part that has seen nothing (m = -inf).
__device__ __forceinline__ float weight_of(float m, float top) {
    return m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - top);
}

}  // namespace w4k
