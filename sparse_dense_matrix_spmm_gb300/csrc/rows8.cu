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
// Vectors of a thread that are loaded before anything is stored.
template <int V>
constexpr int kFlight = V >= 4 ? 4 : 8;

struct Rows8Args {
    void* x;
    int64_t ldx;
    int64_t rows, cols;
    int8_t* q;
    int64_t ldq;
    uint8_t* scale;
    int64_t lds;
    int32_t tx;  // threads along a row, a power of two; kThreads / tx rows per CTA
    bool wide;   // packing: integers leave 4 (fp32) or 8 at a time
};

template <int V>
using Bytes = typename Word<(V < 2 ? 2 : V)>::type;  // V integers as they move (one: a byte of the word)

template <int V>
__device__ __forceinline__ void store_q(int8_t* p, const uint32_t (&q)[V]) {
    static_assert(V == 8 || V == 4, "16 bytes of a row");
    if constexpr (V == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
    else
        *reinterpret_cast<uint32_t*>(p) = pack4(q[0], q[1], q[2], q[3]);
}
template <int V>
__device__ __forceinline__ Bytes<V> load_q(const int8_t* p) {
    if constexpr (V == 1)
        return static_cast<uint8_t>(*p);
    else
        return *reinterpret_cast<const Bytes<V>*>(p);
}

// The largest magnitude's bits among a thread's 16 bytes: magnitudes order as
// integers, NaN above infinity.
template <typename T>
__device__ __forceinline__ uint32_t largest(const uint32_t (&w)[4]) {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return max(m & 0xFFFFu, m >> 16);
    }
}
template <typename T>
__device__ __forceinline__ float of_bits(uint32_t b) {
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(b);
    } else {
        const uint16_t w = static_cast<uint16_t>(b);
        T v;
        memcpy(&v, &w, sizeof(v));
        return to_f32<T>(v);
    }
}

// 16 bytes of a row per thread and vector, loaded in pieces of P values as the
// row's alignment allows; 2 or 4 neighbouring threads per group.  (A value per thread, 16 threads
// per group, for rows without alignment: 12.9 us where this takes 6.5 us, 1537 x 2051 fp32.)
template <typename T, int P>
__global__ void __launch_bounds__(kThreads) pack_kernel(const Rows8Args a) {
    constexpr int V = 16 / static_cast<int>(sizeof(T)), kVecs = 4;
    using X = Vec<T, V>;
    using Piece = Vec<T, P>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int x = threadIdx.x % a.tx, step = a.tx * V;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / a.tx) + threadIdx.x / a.tx;
    const int64_t cols = row < a.rows ? a.cols : 0;
    const bool all_rows = (static_cast<int64_t>(blockIdx.x) + 1) * (kThreads / a.tx) <= a.rows;
    const T* in = static_cast<const T*>(a.x) + row * a.ldx;
    int8_t* q = a.q + row * a.ldq;
    uint8_t* scale = a.scale + row * a.lds;
    // Four vectors of each thread; `whole`: all of them lie in their rows.
    auto turn = [&](int64_t c0, auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        const int64_t c = c0 + x * V;
        uint32_t r[kVecs][4];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            typename Piece::Raw part[V / P];
#pragma unroll
            for (int j = 0; j < V / P; ++j) {
                const int64_t at = c + i * step + j * P;
                part[j] = kWhole || at < cols ? Piece::load(in + at) : Piece::zero();  // cols % P == 0
            }
            memcpy(r[i], part, sizeof(r[i]));
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (!kWhole && c0 + i * step >= a.cols) break;  // alike for all threads
            uint32_t m = largest<T>(r[i]);
#pragma unroll
            for (int d = 1; d < kGroup / V; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
            const uint32_t b = scale_byte(magnitude_code(of_bits<T>(m)));
            const int64_t at = c + i * step;
            typename X::Raw raw;
            memcpy(&raw, r[i], sizeof(raw));
            float f[V];
            X::unpack(raw, f);
            uint32_t v[V];
            quantise(f, b, v);
            if (!kWhole && at >= cols) continue;
            if (a.wide && (kWhole || at + V <= cols)) {
                store_q<V>(q + at, v);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (kWhole || at + j < cols) q[at + j] = static_cast<int8_t>(v[j]);
            }
            if (at % kGroup == 0) scale[at / kGroup] = static_cast<uint8_t>(b);
        }
    };
    for (int64_t c0 = 0; c0 < a.cols; c0 += kVecs * step) {  // whole warps stay together for the shuffles
        if (P == V && all_rows && c0 + kVecs * step <= a.cols)
            turn(c0, std::true_type());
        else
            turn(c0, std::false_type());
    }
}

// fp16: 65536, as which its largest values are held (65024 and more beside one of 65280
// or more), reads back as 65504; what is larger was no fp16 value and becomes infinity.  No
// other multiple of a unit lies between the two.
constexpr uint32_t kHalfTop = 127 + 10;  // scale bytes below have less

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const Rows8Args a) {
    using X = Vec<T, V>;
    constexpr bool kHalf = std::is_same<T, __half>::value;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int x = threadIdx.x % a.tx, step = a.tx * V;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / a.tx) + threadIdx.x / a.tx;
    if (row >= a.rows) return;
    T* out = static_cast<T*>(a.x) + row * a.ldx;
    const int8_t* q = a.q + row * a.ldq;
    const uint8_t* scale = a.scale + row * a.lds;
    for (int64_t c = x * V; c < a.cols; c += kFlight<V> * step) {
        Bytes<V> r[kFlight<V>];
        uint8_t b[kFlight<V>];
#pragma unroll
        for (int i = 0; i < kFlight<V>; ++i) {
            const int64_t at = c + i * step;
            if (at < a.cols) {
                r[i] = load_q<V>(q + at);
                b[i] = scale[at / kGroup];
            }
        }
#pragma unroll
        for (int i = 0; i < kFlight<V>; ++i) {
            const int64_t at = c + i * step;
            if (at >= a.cols) break;
            uint32_t w[2] = {0u, 0u};
            memcpy(w, &r[i], sizeof(r[i]));
            const float unit = unit_of(b[i]);
            float f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = byte_of(w[j >> 2] ^ 0x80808080u, j & 3) * unit;
            if (kHalf && b[i] >= kHalfTop) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (fabsf(f[j]) == 65536.f) f[j] = copysignf(65504.f, f[j]);
            }
            X::store(out + at, X::pack(f));
        }
    }
}

// Whether rows of integers can move n at a time.
bool moves(const spmm_rows8_t* P, int n) {
    return reinterpret_cast<uintptr_t>(P->q) % static_cast<unsigned>(n) == 0 && P->ldq % n == 0;
}

// `per`: values of a thread per turn; `least`: threads of a group.  No more threads to a row than
// have work: short rows share a CTA (61657 x 87 bf16 to 8 bits: 24 us at 16 threads and
// four vectors, 8 us so).
Rows8Args arguments(void* x, int64_t ldx, const spmm_rows8_t* P, int per, int least, dim3& grid) {
    Rows8Args a{x, ldx, P->rows, P->cols, P->q, P->ldq, P->scale, P->lds, least, false};
    while (a.tx < kThreads && a.tx * per < P->cols) a.tx *= 2;
    const int64_t rows = kThreads / a.tx;
    grid = dim3(static_cast<unsigned>((P->rows + rows - 1) / rows));
    return a;
}

}  // namespace

spmm_status launch_pack_rows(const void* x, int64_t ldx, int32_t dtype, const spmm_rows8_t* P, cudaStream_t s) {
    const int es = row_elem_bytes(dtype), p = row_width({Operand{x, ldx, es}}, P->cols);
    dim3 grid;
    Rows8Args a = arguments(const_cast<void*>(x), ldx, P, 4 * 16 / es, es, grid);
    a.wide = moves(P, 16 / es);
    cudaError_t e;
    trace_begin(SPMM_KERNEL_ROWS8, s);
    SPMM_ROWS_TYPED(e, dtype, p, pack_kernel, grid, kThreads, s, a);
    trace_end(SPMM_KERNEL_ROWS8, s);
    return cuda_status(e);
}

spmm_status launch_unpack_rows(const spmm_rows8_t* P, void* out, int64_t ldo, int32_t dtype, cudaStream_t s) {
    int v = row_width({Operand{out, ldo, row_elem_bytes(dtype)}}, P->cols);
    while (v > 1 && !moves(P, v)) v /= 2;
    dim3 grid;
    const Rows8Args a = arguments(out, ldo, P, v * (v >= 4 ? kFlight<4> : kFlight<1>), 1, grid);
    cudaError_t e;
    trace_begin(SPMM_KERNEL_ROWS8, s);
    SPMM_ROWS_TYPED(e, dtype, v, unpack_kernel, grid, kThreads, s, a);
    trace_end(SPMM_KERNEL_ROWS8, s);
    return cuda_status(e);
}

}  // namespace spmm
