// gated.cuh -- device pieces that the gated experts and the 8-bit rows share:
// activations with their derivatives, and groups of 16 values in 8 bits.
#pragma once

#include <cstdint>

#include "spmm_gb300.h"

namespace spmm {
namespace gated {

// act(x), fp32 as CUDA's functions round it.  expf(-x) overflows to infinity for x
// below -88, where silu rounds to -0.
template <int ACT>
__device__ __forceinline__ float act(float x) {
    if (ACT == SPMM_ACT_SILU) return x / (1.f + expf(-x));
    if (ACT == SPMM_ACT_GELU) return 0.5f * x * erfcf(-0.70710678f * x);  // erfc: no cancellation for x < 0
    // (1 + tanh z) / 2 = 1 / (1 + e^-2z), again without cancellation
    const float z = 0.79788456f * (x + 0.044715f * x * x * x);
    return x / (1.f + expf(-2.f * z));
}

// act(x) and its derivative.
template <int ACT>
__device__ __forceinline__ void act_grad(float x, float& f, float& d) {
    if (ACT == SPMM_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-x));
        f = x * s;
        d = s * (1.f + x * (1.f - s));
    } else if (ACT == SPMM_ACT_GELU) {
        const float p = 0.5f * erfcf(-0.70710678f * x);
        f = x * p;
        d = p + x * 0.39894228f * expf(-0.5f * x * x);
    } else {
        const float x2 = x * x, z = 0.79788456f * (x + 0.044715f * x * x2);
        const float s = 1.f / (1.f + expf(-2.f * z));
        const float t = s * (1.f - s);  // 0 where x^2 may overflow
        f = x * s;
        d = t > 0.f ? s + 2.f * x * t * 0.79788456f * (1.f + 0.134145f * x2) : s;
    }
}

// ------------------------------------------------------------------ rows in 8 bits
constexpr int kGroup = 16;
constexpr uint32_t kNotFinite = 511;

// The exponent that a value asks of its group: biased by 127 and rounded up where
// the value is 127.5 / 128 of the next power of two or more (2^16 of the
// significand's 2^23), because it would round to 128.  Monotonic, so a group's
// exponent is the largest of its values'.
__device__ __forceinline__ uint32_t magnitude_code(float x) {
    const uint32_t a = __float_as_uint(x) & 0x7FFFFFFFu;
    return a >= 0x7F800000u ? kNotFinite : (a + 0x10000u) >> 23;
}
// The group's scale byte: magnitudes below 2^(c - 126) less half a step fit
// integers of 127 at 2^(c - 133).
__device__ __forceinline__ uint32_t scale_byte(uint32_t code) {
    if (code == kNotFinite) return 255u;
    const int b = static_cast<int>(code) - 6;
    return static_cast<uint32_t>(b < 1 ? 1 : b > 248 ? 248 : b);
}
// x in units of the scale: exact but for the one rounding (a power of two).
__device__ __forceinline__ int quantise(float x, uint32_t byte) {
    if (byte == 255u) return 0;
    const int q = __float2int_rn(x * __uint_as_float((254u - byte) << 23));
    return q > 127 ? 127 : q < -127 ? -127 : q;
}
// 2^e; infinity for 255, which makes NaN of the q = 0 beside it.
__device__ __forceinline__ float unit_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four integers as bytes, and back.
__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (static_cast<uint32_t>(a) & 255u) | ((static_cast<uint32_t>(b) & 255u) << 8) |
           ((static_cast<uint32_t>(c) & 255u) << 16) | (static_cast<uint32_t>(d) << 24);
}
__device__ __forceinline__ int byte_of(uint32_t w, int i) {
    return static_cast<int>(static_cast<int8_t>(w >> (8 * i)));
}

}  // namespace gated
}  // namespace spmm
