// gated.cuh -- device pieces that the gated experts and the 8-bit rows share:
// activations with their derivatives, and groups of 16 values in 8 bits.
#pragma once

#include <cstdint>

#include "spmm_gb300.h"

namespace spmm {
namespace gated {

// 1 / (1 + 2^x).  Both instructions are off by a unit or two of 2^-23, and a rounded x
// by |x| 2^-24 of the power: below 2^-19 for |x| <= 16, where results round to 2^-9 or 2^-12.
// Their .ftz forms spare the handling of subnormal numbers, whose results round to 0 or 1
// here: with expf and an exact division the gradient of the activation took 47 us where
// it takes 31 us (16372 x 1280, silu), bound by instructions.
__device__ __forceinline__ float over_1_plus_exp2(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
constexpr float kLog2e = 1.44269504f;
// silu: x / (1 + 2^(-x log2 e)).  Tanh form: (1 + tanh z) / 2 = 1 / (1 + 2^(-2 z log2 e)) with
// 2 z = x (kTanh + kTanh3 x^2), kTanh = 2 sqrt(2 / pi), kTanh3 = 0.044715 kTanh.
constexpr float kTanh = 1.59576912f, kTanh3 = 0.0713548163f;
__device__ __forceinline__ float gate_of_tanh(float x, float x2) {
    return over_1_plus_exp2(x * fmaf(-kTanh3 * kLog2e, x2, -kTanh * kLog2e));
}

// act(x); gelu by erfc (no cancellation for x < 0).
template <int ACT>
__device__ __forceinline__ float act(float x) {
    if (ACT == SPMM_ACT_SILU) return x * over_1_plus_exp2(-kLog2e * x);
    if (ACT == SPMM_ACT_GELU) return 0.5f * x * erfcf(-0.70710678f * x);
    return x * gate_of_tanh(x, x * x);
}

// act(x) and its derivative.
template <int ACT>
__device__ __forceinline__ void act_grad(float x, float& f, float& d) {
    if (ACT == SPMM_ACT_SILU) {
        const float s = over_1_plus_exp2(-kLog2e * x);
        f = x * s;
        d = fmaf(f, 1.f - s, s);
    } else if (ACT == SPMM_ACT_GELU) {
        const float p = 0.5f * erfcf(-0.70710678f * x);
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-0.5f * kLog2e * x * x));
        f = x * p;
        d = fmaf(0.39894228f * x, e, p);
    } else {
        const float x2 = fminf(x * x, 1e30f);  // finite: it meets s (1 - s) = 0 below
        const float s = gate_of_tanh(x, x2);
        f = x * s;
        d = fmaf(f * (1.f - s), fmaf(3.f * kTanh3, x2, kTanh), s);
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
// Values in units of the scale, exact but for the one rounding (a power of two):
// words whose lowest bytes are the integers.  The sum with 1.5 2^23 leaves no bits below
// the units, so it is rounded there, half to even.  Scales next to the type's largest
// values cut off at 127, and a group that is not finite is zeros.
template <int V>
__device__ __forceinline__ void quantise(const float (&x)[V], uint32_t byte, uint32_t (&q)[V]) {
    const float inverse = __uint_as_float((254u - byte) << 23);
    if (byte < 248u) {
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = __float_as_uint(fmaf(x[i], inverse, 12582912.f));
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = __float2int_rn(x[i] * inverse);
        q[i] = byte == 255u ? 0u : static_cast<uint32_t>(v > 127 ? 127 : v < -127 ? -127 : v);
    }
}
// 2^e; infinity for 255, which makes NaN of the q = 0 beside it.
__device__ __forceinline__ float unit_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// The lowest bytes of four words.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Signed byte i of a word whose bytes have 128 added (w ^ 0x80808080), as fp32: the
// byte in the last place of 2^23, less that.
__device__ __forceinline__ float byte_of(uint32_t w, int i) {
    return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | static_cast<uint32_t>(i))) - 8388736.f;
}

}  // namespace gated
}  // namespace spmm
