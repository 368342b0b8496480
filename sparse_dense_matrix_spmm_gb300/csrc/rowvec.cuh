// rowvec.cuh -- row elements as fp32 vectors: loads, stores and conversions
// shared by the one-hot row operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace spmm {
namespace rows {

// One value to and from fp32 (round to nearest even).
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two packed 16-bit values.
template <typename T>
struct Pair;
template <>
struct Pair<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t v) {  // a bf16 is the high half of an fp32
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// V consecutive elements of type T: V = 16 / sizeof(T) moves 16 bytes at once
// (the address must be 16-byte aligned), V = 1 one element.
template <typename T, int V>
struct Vec {
    using Raw = uint4;
    static __device__ __forceinline__ Raw load(const T* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
    // data read once: leaves the caches first
    static __device__ __forceinline__ Raw load_cs(const T* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
    static __device__ __forceinline__ void store(T* p, const Raw& r) { *reinterpret_cast<uint4*>(p) = r; }
    static __device__ __forceinline__ void store_cs(T* p, const Raw& r) { __stcs(reinterpret_cast<uint4*>(p), r); }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[V]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                const float2 p = Pair<T>::unpack(w[i]);
                f[2 * i] = p.x;
                f[2 * i + 1] = p.y;
            }
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[V]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(f[i]);
            else
                w[i] = Pair<T>::pack(f[2 * i], f[2 * i + 1]);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <typename T>
struct Vec<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ Raw load(const T* p) { return __ldg(p); }
    static __device__ __forceinline__ Raw load_cs(const T* p) { return __ldg(p); }
    static __device__ __forceinline__ void store(T* p, const Raw& r) { *p = r; }
    static __device__ __forceinline__ void store_cs(T* p, const Raw& r) { *p = r; }
    static __device__ __forceinline__ Raw zero() { return from_f32<T>(0.f); }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[1]) { f[0] = to_f32<T>(r); }
    static __device__ __forceinline__ Raw pack(const float (&f)[1]) { return from_f32<T>(f[0]); }
};

// Four 16-bit values next to four fp32 ones: 8 bytes at once.
template <typename T>
struct Vec4x16 {
    using Raw = uint2;
    static __device__ __forceinline__ void store_cs(T* p, const Raw& r) { __stcs(reinterpret_cast<uint2*>(p), r); }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[4]) {
        const float2 a = Pair<T>::unpack(r.x), b = Pair<T>::unpack(r.y);
        f[0] = a.x;
        f[1] = a.y;
        f[2] = b.x;
        f[3] = b.y;
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[4]) {
        return make_uint2(Pair<T>::pack(f[0], f[1]), Pair<T>::pack(f[2], f[3]));
    }
};
template <>
struct Vec<__half, 4> : Vec4x16<__half> {};
template <>
struct Vec<__nv_bfloat16, 4> : Vec4x16<__nv_bfloat16> {};

// Eight fp32 values next to eight 16-bit ones: 32 bytes as two 16-byte moves.
template <>
struct Vec<float, 8> {
    struct Raw {
        uint4 lo, hi;
    };
    static __device__ __forceinline__ Raw load(const float* p) {
        return {__ldg(reinterpret_cast<const uint4*>(p)), __ldg(reinterpret_cast<const uint4*>(p) + 1)};
    }
    static __device__ __forceinline__ void store(float* p, const Raw& r) {
        reinterpret_cast<uint4*>(p)[0] = r.lo;
        reinterpret_cast<uint4*>(p)[1] = r.hi;
    }
    static __device__ __forceinline__ void store_cs(float* p, const Raw& r) {
        __stcs(reinterpret_cast<uint4*>(p), r.lo);
        __stcs(reinterpret_cast<uint4*>(p) + 1, r.hi);
    }
    static __device__ __forceinline__ Raw zero() { return {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[8]) {
        const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[8]) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
        return {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
    }
};

}  // namespace rows

// Rows move in 16-byte pieces when the base, the pitch and the row length are
// all multiples of 16 bytes, else one element at a time.
inline bool rows16(const void* p, int64_t ld, int64_t H, int es) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0 && (H * es) % 16 == 0;
}

}  // namespace spmm

// Threads of a CTA that moves rows of H elements, V at a time.
inline int row_threads(int64_t H, int V, int most) {
    const int64_t n = ((H + V - 1) / V + 31) / 32 * 32;
    return static_cast<int>(n < most ? n : most);
}

// Launch KERNEL<T, V> for a row type and vector width chosen at run time.
#define SPMM_ROWS_TYPED(status, dtype, vec, KERNEL, grid, threads, s, args)                                      \
    do {                                                                                                         \
        if ((dtype) == SPMM_F32)                                                                                 \
            status = launch_chained(vec ? KERNEL<float, 4> : KERNEL<float, 1>, grid, threads, 0, 1, s, args);    \
        else if ((dtype) == SPMM_F16)                                                                            \
            status = launch_chained(vec ? KERNEL<__half, 8> : KERNEL<__half, 1>, grid, threads, 0, 1, s, args);  \
        else                                                                                                     \
            status = launch_chained(vec ? KERNEL<__nv_bfloat16, 8> : KERNEL<__nv_bfloat16, 1>, grid, threads, 0, \
                                    1, s, args);                                                                 \
    } while (0)
