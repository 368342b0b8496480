// rows8.cu -- rows held in 8 bits and read back: groups of 16 values of a row share
// a power of two, the smallest for which all of them round to integers of at most
// 127.  Both directions are bound by HBM (2 + 17/16 bytes a value for 16-bit rows).
// A power of two makes scaling exact, so a value is rounded once and a checkpoint's bits
// depend on the values alone; its exponent comes from the bits of the largest magnitude,
// without a division.
#include "gated.cuh"
#include "internal.h"
#include "rowvec.cuh"

namespace spmm {
namespace {

using namespace rows;
using namespace gated;

constexpr int kThreads = 256;

struct Rows8Args {
    void* x;
    int64_t ldx;
    int64_t rows, cols;
    int8_t* q;
    int64_t ldq;
    uint8_t* scale;
    int64_t lds;
    int32_t tx;  // threads along a row, a power of two of at least 16; blockDim / tx rows per CTA
};

template <int V>
__device__ __forceinline__ void store_q(int8_t* p, const int (&q)[V]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
    else if constexpr (V == 4)
        *reinterpret_cast<uint32_t*>(p) = pack4(q[0], q[1], q[2], q[3]);
    else if constexpr (V == 2)
        *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(pack4(q[0], q[1], 0, 0));
    else
        *p = static_cast<int8_t>(q[0]);
}
template <int V>
__device__ __forceinline__ void load_q(const int8_t* p, int (&q)[V]) {
    uint32_t w[2] = {0u, 0u};
    if constexpr (V == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else if constexpr (V == 4) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (V == 2) {
        w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
        w[0] = static_cast<uint8_t>(*p);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = byte_of(w[i >> 2], i & 3);
}

// V values per thread, 16 / V neighbouring threads per group.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) pack_kernel(const Rows8Args a) {
    using X = Vec<T, V>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int x = threadIdx.x % a.tx;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.tx) + threadIdx.x / a.tx;
    const bool live = row < a.rows;
    const T* in = static_cast<const T*>(a.x) + row * a.ldx;
    int8_t* q = a.q + row * a.ldq;
    uint8_t* scale = a.scale + row * a.lds;
    for (int64_t c0 = 0; c0 < a.cols; c0 += a.tx * V) {  // whole warps stay together for the shuffles
        const int64_t c = c0 + x * V;
        const bool in_row = live && c < a.cols;
        float f[V];
        X::unpack(in_row ? X::load(in + c) : X::zero(), f);
        uint32_t code = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) code = max(code, magnitude_code(f[i]));
#pragma unroll
        for (int d = 1; d < kGroup / V; d <<= 1) code = max(code, __shfl_xor_sync(0xffffffffu, code, d));
        const uint32_t b = scale_byte(code);
        if (!in_row) continue;
        int v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = quantise(f[i], b);
        store_q<V>(q + c, v);
        if (c % kGroup == 0) scale[c / kGroup] = static_cast<uint8_t>(b);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const Rows8Args a) {
    using X = Vec<T, V>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int x = threadIdx.x % a.tx;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.tx) + threadIdx.x / a.tx;
    if (row >= a.rows) return;
    T* out = static_cast<T*>(a.x) + row * a.ldx;
    const int8_t* q = a.q + row * a.ldq;
    const uint8_t* scale = a.scale + row * a.lds;
    for (int64_t c = x * V; c < a.cols; c += a.tx * V) {
        int v[V];
        load_q<V>(q + c, v);
        const float unit = unit_of(scale[c / kGroup]);
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = static_cast<float>(v[i]) * unit;
        X::store(out + c, X::pack(f));
    }
}

// The widest move that rows and integers allow.
int width_of(const void* x, int64_t ldx, int32_t dtype, const spmm_rows8_t* P) {
    const int es = row_elem_bytes(dtype);
    int v = row_width({Operand{x, ldx, es}}, P->cols);
    while (v > 1 && (reinterpret_cast<uintptr_t>(P->q) % static_cast<unsigned>(v) || P->ldq % v)) v /= 2;
    return v;
}

Rows8Args arguments(void* x, int64_t ldx, const spmm_rows8_t* P, int v, dim3& grid) {
    Rows8Args a{x, ldx, P->rows, P->cols, P->q, P->ldq, P->scale, P->lds, 16};
    while (a.tx < kThreads && a.tx * v < P->cols) a.tx *= 2;
    const int64_t per = kThreads / a.tx;
    grid = dim3(static_cast<unsigned>((P->rows + per - 1) / per));
    return a;
}

}  // namespace

spmm_status launch_pack_rows(const void* x, int64_t ldx, int32_t dtype, const spmm_rows8_t* P, cudaStream_t s) {
    const int v = width_of(x, ldx, dtype, P);
    dim3 grid;
    const Rows8Args a = arguments(const_cast<void*>(x), ldx, P, v, grid);
    cudaError_t e;
    trace_begin(SPMM_KERNEL_ROWS8, s);
    SPMM_ROWS_TYPED(e, dtype, v, pack_kernel, grid, kThreads, s, a);
    trace_end(SPMM_KERNEL_ROWS8, s);
    return cuda_status(e);
}

spmm_status launch_unpack_rows(const spmm_rows8_t* P, void* out, int64_t ldo, int32_t dtype, cudaStream_t s) {
    const int v = width_of(out, ldo, dtype, P);
    dim3 grid;
    const Rows8Args a = arguments(out, ldo, P, v, grid);
    cudaError_t e;
    trace_begin(SPMM_KERNEL_ROWS8, s);
    SPMM_ROWS_TYPED(e, dtype, v, unpack_kernel, grid, kThreads, s, a);
    trace_end(SPMM_KERNEL_ROWS8, s);
    return cuda_status(e);
}

}  // namespace spmm
