// rowvec.cuh -- row elements as fp32 vectors: loads, stores and conversions
// shared by the one-hot row operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "sm103_more.cuh"

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

// Words that move at once.
template <int BYTES>
struct Word;
template <>
struct Word<2> {
    using type = uint16_t;
};
template <>
struct Word<4> {
    using type = uint32_t;
};
template <>
struct Word<8> {
    using type = uint2;
};
template <>
struct Word<16> {
    using type = uint4;
};

// V consecutive elements of type T, V sizeof(T) = 2, 4, 8 or 16 bytes moved at
// once (32 bytes, eight fp32 next to eight 16-bit values, in two halves).  The
// address must be a multiple of those bytes (of 16 for 32).
template <typename T, int V>
struct Vec {
    static constexpr int kBytes = V * static_cast<int>(sizeof(T)), kWords = (kBytes + 15) / 16;
    using W = typename Word<(kBytes < 16 ? kBytes : 16)>::type;
    struct Two {
        W w[2];
    };
    using Raw = std::conditional_t<kWords == 1, W, Two>;
    static __device__ __forceinline__ W* words(Raw& r) { return reinterpret_cast<W*>(&r); }
    static __device__ __forceinline__ const W* words(const Raw& r) { return reinterpret_cast<const W*>(&r); }
    static __device__ __forceinline__ Raw load(const T* p) {
        Raw r;
#pragma unroll
        for (int i = 0; i < kWords; ++i) words(r)[i] = reinterpret_cast<const W*>(p)[i];
        return r;
    }
    // data read once: leaves the caches first
    static __device__ __forceinline__ Raw load_cs(const T* p) {
        Raw r;
#pragma unroll
        for (int i = 0; i < kWords; ++i) words(r)[i] = ptx::ld_global_cs(reinterpret_cast<const W*>(p) + i);
        return r;
    }
    static __device__ __forceinline__ void store(T* p, const Raw& r) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) reinterpret_cast<W*>(p)[i] = words(r)[i];
    }
    static __device__ __forceinline__ void store_cs(T* p, const Raw& r) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) __stcs(reinterpret_cast<W*>(p) + i, words(r)[i]);
    }
    static __device__ __forceinline__ Raw zero() {
        Raw r;
        memset(&r, 0, sizeof(r));
        return r;
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[V]) {
        if constexpr (sizeof(T) == 4) {
            memcpy(f, &r, sizeof(f));
        } else if constexpr (V == 1) {
            T v;
            memcpy(&v, &r, sizeof(v));
            f[0] = to_f32<T>(v);
        } else {
            uint32_t w[V / 2];
            memcpy(w, &r, sizeof(w));
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 p = Pair<T>::unpack(w[i]);
                f[2 * i] = p.x;
                f[2 * i + 1] = p.y;
            }
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[V]) {
        Raw r;
        if constexpr (sizeof(T) == 4) {
            memcpy(&r, f, sizeof(f));
        } else if constexpr (V == 1) {
            const T v = from_f32<T>(f[0]);
            memcpy(&r, &v, sizeof(v));
        } else {
            uint32_t w[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = Pair<T>::pack(f[2 * i], f[2 * i + 1]);
            memcpy(&r, w, sizeof(w));
        }
        return r;
    }
};

// A thread's columns of a row: U vectors of V elements, `step` columns apart: at
// full width WIDE, in narrower moves as many as make 16 bytes, four at most, times
// DEPTH, so that they too have many bytes in flight.  They are loaded before
// anything is stored (the compiler may not move an ordinary load over a store) and
// without a test each where all of them count.  8192 x 4 x 4095 bf16, dispatch: 107
// us with one at a time, 77 us with four; 16384 tokens, embed: 124 us with one, 65
// us with four, 57 us with eight.  Column c + u step of vector u counts if it lies
// below H.
template <typename T, int V, int WIDE = 1, int DEPTH = 1>
struct Cols {
    static constexpr int kVecs = 16 / (V * static_cast<int>(sizeof(T)));
    static constexpr int U = kVecs == 1 ? WIDE : (kVecs < 4 ? kVecs : 4) * DEPTH, N = U * V;
    using X = Vec<T, V>;
    using Raw = typename X::Raw;
    static __device__ __forceinline__ void load(Raw (&r)[U], const T* row, int64_t c, int64_t H, int step) {
        if (c + (U - 1) * step < H) {
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = X::load(row + c + u * step);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = c + u * step < H ? X::load(row + c + u * step) : X::zero();
        }
    }
    static __device__ __forceinline__ void clear(Raw (&r)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = X::zero();
    }
    static __device__ __forceinline__ void store(T* row, const Raw (&r)[U], int64_t c, int64_t H, int step) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * step < H) X::store(row + c + u * step, r[u]);
    }
    static __device__ __forceinline__ void store_cs(T* row, const Raw (&r)[U], int64_t c, int64_t H, int step) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * step < H) X::store_cs(row + c + u * step, r[u]);
    }
    static __device__ __forceinline__ void unpack(const Raw (&r)[U], float (&f)[N]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[V];
            X::unpack(r[u], v);
#pragma unroll
            for (int i = 0; i < V; ++i) f[u * V + i] = v[i];
        }
    }
    static __device__ __forceinline__ void pack(Raw (&r)[U], const float (&f)[N]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = f[u * V + i];
            r[u] = X::pack(v);
        }
    }
};

}  // namespace rows

// Whether rows of H elements of `es` bytes move V elements at a time.
inline bool rows_move(const void* p, int64_t ld, int64_t H, int es, int V) {
    const int bytes = V * es < 16 ? V * es : 16;
    return reinterpret_cast<uintptr_t>(p) % static_cast<unsigned>(bytes) == 0 && (ld * es) % bytes == 0 && H % V == 0;
}

// Elements per move that the base, pitch and row length of every operand allow,
// 16 bytes at most.  What a width costs, 8192 tokens x 4 in bf16, microseconds:
//   row length      4096 (16 B)  4100 (8 B)  4098 (4 B)  4095 (2 B)
//   dispatch          52           54          64          77
//   combine           51           55          58          76
//   its gradient      92           97         105         137
//   embed, 16384      41           43          45          57
struct Operand {
    const void* p;
    int64_t ld;
    int es;
};
template <int N>
int row_width(const Operand (&o)[N], int64_t H) {
    for (int v = 16 / o[0].es; v > 1; v /= 2) {
        bool ok = true;
        for (const Operand& x : o) ok = ok && rows_move(x.p, x.ld, H, x.es, v);
        if (ok) return v;
    }
    return 1;
}

// Threads of a CTA that moves rows of H elements, `per` of them each; at least a warp.
inline int row_threads(int64_t H, int per, int most) {
    const int64_t n = H ? ((H + per - 1) / per + 31) / 32 * 32 : 32;
    return static_cast<int>(n < most ? n : most);
}

}  // namespace spmm

// Launch KERNEL<T, V> for a row type and vector width (elements) chosen at run time.
#define SPMM_ROWS_TYPED(status, dtype, v, KERNEL, grid, threads, s, args)                                          \
    do {                                                                                                           \
        if ((dtype) == SPMM_F32)                                                                                   \
            status = launch_chained((v) == 4 ? KERNEL<float, 4> : (v) == 2 ? KERNEL<float, 2> : KERNEL<float, 1>,  \
                                    grid, threads, 0, 1, s, args);                                                 \
        else if ((dtype) == SPMM_F16)                                                                              \
            status = launch_chained((v) == 8   ? KERNEL<__half, 8>                                                 \
                                    : (v) == 4 ? KERNEL<__half, 4>                                                 \
                                    : (v) == 2 ? KERNEL<__half, 2>                                                 \
                                               : KERNEL<__half, 1>,                                                \
                                    grid, threads, 0, 1, s, args);                                                 \
        else                                                                                                       \
            status = launch_chained((v) == 8   ? KERNEL<__nv_bfloat16, 8>                                          \
                                    : (v) == 4 ? KERNEL<__nv_bfloat16, 4>                                          \
                                    : (v) == 2 ? KERNEL<__nv_bfloat16, 2>                                          \
                                               : KERNEL<__nv_bfloat16, 1>,                                         \
                                    grid, threads, 0, 1, s, args);                                                 \
    } while (0)
