// Device side of the 8-bit checkpoint format: e4m3 codes and a power-of-two scale byte for each 32 values of
// a row.
//
// The scale of a block is 2^e with the smallest e >= -120 for which amax <= 448 * 2^e.  448 = 1.75 * 2^8, so
// with amax = m * 2^k (m in [1, 2)) e is k - 8, or k - 7 where m > 1.75: adding 0x1fffff to the bits of amax
// carries into the exponent field exactly for a fraction above 0.75, and the scale byte e + 127 is that field
// less 8.  e >= -120 keeps the smallest step, 2^(e - 9), exact in bf16.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kCkptBlock = 32;
constexpr uint32_t kInfBits = 0x7f800000u;
// 240 * 2^120: magnitudes above this would round to 256 * 2^120, which is infinity
constexpr uint32_t kCkptTopBits = 0x7ff00000u - 0x00800000u;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// The magnitude's bits where it is finite, else 0 (such a value has no part in its block's scale).
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
    const uint32_t b = abs_bits(x);
    return b < kInfBits ? b : 0u;
}

// Scale byte of a block from the bits of its largest finite magnitude.
__device__ __forceinline__ int ckpt_scale(uint32_t amax_bits) {
    const int field = (int)((amax_bits + 0x1fffffu) >> 23) - 8;
    return field < 7 ? 7 : field;
}
// 2^-e for scale bytes that ckpt_scale gives (7 .. 247), and 2^e for bytes up to 254.
__device__ __forceinline__ float ckpt_inverse(int scale) { return __uint_as_float((uint32_t)(254 - scale) << 23); }
__device__ __forceinline__ float ckpt_unit(int scale) { return __builtin_amdgcn_ldexpf(1.f, scale - 127); }

// Codes of a and b, scaled, in the low or the high half of `into` (round to nearest even).
template <bool HIGH>
__device__ __forceinline__ uint32_t ckpt_code2(float a, float b, float inv, uint32_t into) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, (int)into, HIGH);
}
// The code of any value: infinities and NaN give the NaN code, magnitudes at the type's top are cut.
__device__ __forceinline__ uint32_t ckpt_code_any(float x, float inv) {
    if (abs_bits(x) >= kInfBits) return 0x7f;
    const float top = __uint_as_float(kCkptTopBits);
    return ckpt_code2<false>(__builtin_amdgcn_fmed3f(x, -top, top), 0.f, inv, 0) & 0xff;
}
// Four codes in a word; `any`: the block holds values that need ckpt_code_any.
__device__ __forceinline__ uint32_t ckpt_code4(const float* x, float inv, bool any) {
    if (any)
        return ckpt_code_any(x[0], inv) | ckpt_code_any(x[1], inv) << 8 | ckpt_code_any(x[2], inv) << 16 |
               ckpt_code_any(x[3], inv) << 24;
    return ckpt_code2<true>(x[2], x[3], inv, ckpt_code2<false>(x[0], x[1], inv, 0));
}
// Four values of a word of codes, unit = 2^e.
__device__ __forceinline__ void ckpt_value4(uint32_t codes, float unit, float* x) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
    x[0] = lo[0] * unit; x[1] = lo[1] * unit; x[2] = hi[0] * unit; x[3] = hi[1] * unit;
}

// Largest magnitude's bits of N values (above kCkptTopBits where one is not finite), and of the finite ones only.
template <int N>
__device__ __forceinline__ uint32_t ckpt_amax(const float* x) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) m = max(m, abs_bits(x[k]));
    return m;
}
template <int N>
__device__ __forceinline__ uint32_t ckpt_amax_finite(const float* x) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) m = max(m, finite_abs_bits(x[k]));
    return m;
}

// The largest over groups of LANES neighbouring lanes, in each of them (1, 2, 4, 8, 16 or 32; all lanes of a group
// active).
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LANES >= 2) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));    // lane ^ 1
    if constexpr (LANES >= 4) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));    // lane ^ 2
    if constexpr (LANES >= 8) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));   // mirrored 8
    if constexpr (LANES >= 16) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));  // mirrored 16
    if constexpr (LANES >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    return v;
}

// Scale byte of a block that LANES lanes share, N values in each (`in`: this lane's are part of it), and whether its codes
// need ckpt_code_any.
template <int LANES, int N>
__device__ __forceinline__ int ckpt_block(const float* x, bool in, bool& any) {
    uint32_t top = lanes_max<LANES>(in ? ckpt_amax<N>(x) : 0);
    any = top > kCkptTopBits;
    if (any) top = lanes_max<LANES>(in ? ckpt_amax_finite<N>(x) : 0);
    return ckpt_scale(top);
}

}  // namespace kda
