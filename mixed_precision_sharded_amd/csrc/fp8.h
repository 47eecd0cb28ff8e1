// The 8-bit block format's device arithmetic: the scale byte of a run of 32
// elements, and the conversions between values and codes.  Shared by the
// 8-bit moment state (kernels_q8.hip) and the 8-bit activations.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace mps {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Largest finite code of each format is 1.75 * 2^k: 448 (E4M3), 57344 (E5M2).
constexpr int kE4M3TopExp = 8;
constexpr int kE5M2TopExp = 15;
constexpr uint32_t kNonFinite = 255;

// ------------------------------------------------------ scales and codes ---

// 2^(byte - 127); byte 0 is the subnormal 2^-127; 255 gives NaN.
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    uint32_t bits = byte << 23;
    bits = byte == 0 ? 0x00400000u : bits;
    bits = byte == kNonFinite ? 0x7fc00000u : bits;
    return __uint_as_float(bits);
}

// The scale byte of a run whose largest magnitude has the bit pattern
// `absbits` (sign cleared): the smallest e >= -127 with
// absmax <= 1.75 * 2^(kTopExp + e), or 255 when the run is not finite.
template <int kTopExp>
__device__ __forceinline__ uint32_t scale_byte(uint32_t absbits)
{
    if (absbits >= 0x7f800000u) return kNonFinite;
    int e = static_cast<int>(absbits >> 23) - 127 - kTopExp + ((absbits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < -127 ? -127 : e;
    return static_cast<uint32_t>(e + 127);
}

// 2^-e for a finite scale byte (exact: e <= 120 for any finite fp32 run).
__device__ __forceinline__ float inverse_scale(uint32_t byte)
{
    return __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The two codes in the low (kHigh false) or high half of `word`, widened.
template <bool kE4M3, bool kHigh>
__device__ __forceinline__ f32x2 decode_pair(uint32_t word)
{
    return kE4M3 ? __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(word), kHigh)
                 : __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(word), kHigh);
}

// Four codes (one word) to values times `scale`.
template <bool kE4M3>
__device__ __forceinline__ void decode4(uint32_t codes, float scale, float (&out)[4])
{
    const f32x2 lo = decode_pair<kE4M3, false>(codes);
    const f32x2 hi = decode_pair<kE4M3, true>(codes);
    out[0] = lo[0] * scale;
    out[1] = lo[1] * scale;
    out[2] = hi[0] * scale;
    out[3] = hi[1] * scale;
}

// Round a and b to codes (nearest, ties to even) into the low (kHigh false)
// or high half of `old`, keeping the other half.
template <bool kE4M3, bool kHigh>
__device__ __forceinline__ uint32_t encode_pair(float a, float b, uint32_t old)
{
    return static_cast<uint32_t>(kE4M3 ? __builtin_amdgcn_cvt_pk_fp8_f32(a, b, static_cast<int>(old), kHigh)
                                       : __builtin_amdgcn_cvt_pk_bf8_f32(a, b, static_cast<int>(old), kHigh));
}

// Four values to codes at the run's scale byte (all 0xFF for a non-finite
// run).
template <bool kE4M3>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], uint32_t byte)
{
    const float inv = inverse_scale(byte);
    uint32_t word = encode_pair<kE4M3, false>(x[0] * inv, x[1] * inv, 0u);
    word = encode_pair<kE4M3, true>(x[2] * inv, x[3] * inv, word);
    return byte == kNonFinite ? 0xffffffffu : word;
}

template <bool kE4M3>
__device__ __forceinline__ uint32_t encode1(float x, uint32_t byte)
{
    const uint32_t word = encode_pair<kE4M3, false>(x * inverse_scale(byte), 0.0f, 0u);
    return byte == kNonFinite ? 0xffu : (word & 0xffu);
}

template <bool kE4M3>
__device__ __forceinline__ float decode1(uint32_t code, float scale)
{
    return decode_pair<kE4M3, false>(code)[0] * scale;
}

}  // namespace
}  // namespace mps
