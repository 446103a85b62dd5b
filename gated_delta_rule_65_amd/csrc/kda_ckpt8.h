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
// 2^-e for scale bytes that ckpt_scale gives (7 .. 247).
__device__ __forceinline__ float ckpt_inverse(int scale) { return __uint_as_float((uint32_t)(254 - scale) << 23); }

// A finite value ready for the conversion: scaled, and no larger than what unpacks to a finite value.
__device__ __forceinline__ float ckpt_scaled(float x, float inv) {
    const float top = __uint_as_float(kCkptTopBits);
    return __builtin_amdgcn_fmed3f(x, -top, top) * inv;
}
// Codes of a and b in the low 16 bits (round to nearest even); infinities and NaN give the NaN code.
__device__ __forceinline__ uint32_t ckpt_code2(float a, float b, float inv) {
    uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(ckpt_scaled(a, inv), ckpt_scaled(b, inv), 0, false) & 0xffffu;
    if (abs_bits(a) >= kInfBits) c |= 0x7fu;
    if (abs_bits(b) >= kInfBits) c |= 0x7f00u;
    return c;
}
// The value of byte `sel` of `codes` under a scale byte (any byte).
template <int SEL>
__device__ __forceinline__ float ckpt_value(uint32_t codes, int scale) {
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_cvt_f32_fp8((int)codes, SEL), scale - 127);
}

}  // namespace kda
