// gated.cuh -- device pieces that the gated experts and the 8-bit rows share:
// activations with their derivatives, and groups of 16 values in 8 bits.
#pragma once

#include <cstdint>

#include "spmm_gb300.h"

namespace spmm {
namespace gated {

// 2^x and 1 / x, off by a unit or two of 2^-23.  What is rounded in a power's argument comes
// on top: relative to themselves silu's factor is off by 2^-20 + 1.6 |x| 2^-24 at most, Phi by
// 2^-19 + 1.4 x^2 2^-24, the tanh form's factor by 2^-20 + 4 (1.6 |x| + 0.072 |x|^3) 2^-24, where
// results round to 2^-9 or 2^-12.  Their .ftz forms spare the handling of subnormal numbers:
// powers below 2^-126 are 0, and so is act(x) where it is smaller than about 2^-119.
// With expf, erfcf and exact divisions the gradient of the activation took 47 us where
// it takes 31 us (16372 x 1280, silu), bound by instructions.
__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float one_over(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.44269504f;
// silu: x / (1 + 2^(-x log2 e)).  Tanh form: (1 + tanh z) / 2 = 1 / (1 + 2^(-2 z log2 e)) with
// 2 z = x (kTanh + kTanh3 x^2), kTanh = 2 sqrt(2 / pi), kTanh3 = 0.044715 kTanh.
constexpr float kTanh = 1.59576912f, kTanh3 = 0.0713548163f;
__device__ __forceinline__ float gate_of_tanh(float x, float x2) {
    return one_over(1.f + exp2_of(x * fmaf(-kTanh3 * kLog2e, x2, -kTanh * kLog2e)));
}
// The normal distribution function and e = e^(-x^2 / 2).  Phi(-a) = e t R(t) with t =
// 1 / (1 + 0.325 a) for a >= 0; R is a polynomial fitted to Phi(-a) e^(a^2 / 2) / t
// over all of them, off by 6.9e-7 of the value at most, so that nothing cancels for x <
// 0.  (By erfcf the forward pass of 8192 rows, 2 x 1024 x 256, took 28 us, 19 so.)
__device__ __forceinline__ float phi_of(float x, float& e) {
    e = exp2_of(-0.5f * kLog2e * x * x);
    const float t = one_over(fmaf(0.325f, fabsf(x), 1.f));
    float r = 0.0338469292f;
    r = fmaf(r, t, -0.113611606f);
    r = fmaf(r, t, 0.0854171443f);
    r = fmaf(r, t, 0.0259835616f);
    r = fmaf(r, t, 0.0935345683f);
    r = fmaf(r, t, 0.115501354f);
    r = fmaf(r, t, 0.129672222f);
    r = fmaf(r, t, 0.129656151f);
    const float below = e * (t * r);
    return x > 0.f ? 1.f - below : below;
}

// act(x).
template <int ACT>
__device__ __forceinline__ float act(float x) {
    if (ACT == SPMM_ACT_SILU) return x * one_over(1.f + exp2_of(-kLog2e * x));
    if (ACT == SPMM_ACT_GELU) {
        float e;
        return x * phi_of(x, e);
    }
    return x * gate_of_tanh(x, x * x);
}

// act(x) and its derivative.
template <int ACT>
__device__ __forceinline__ void act_grad(float x, float& f, float& d) {
    if (ACT == SPMM_ACT_SILU) {
        const float s = one_over(1.f + exp2_of(-kLog2e * x));
        f = x * s;
        d = fmaf(f, 1.f - s, s);
    } else if (ACT == SPMM_ACT_GELU) {
        float e;
        const float p = phi_of(x, e);
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
// The same from the upper half of a magnitude's bits, which is all that it goes by.
__device__ __forceinline__ uint32_t code_of_upper(uint32_t half) {
    return half >= 0x7F80u ? kNotFinite : (half + 1u) >> 7;
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
constexpr float kRoundUnits = 12582912.f;
template <int V>
__device__ __forceinline__ void quantise(const float (&x)[V], uint32_t byte, uint32_t (&q)[V]) {
    const float inverse = __uint_as_float((254u - byte) << 23);
    if (byte < 248u) {
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = __float_as_uint(fmaf(x[i], inverse, kRoundUnits));
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
