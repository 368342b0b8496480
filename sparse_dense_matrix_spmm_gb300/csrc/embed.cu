// embed.cu -- embedding lookup and its gradient: products with the T x V one-hot
// matrix of token ids.
//   lookup    out    = scale P table          (out[t] = scale table[ids[t]])
//   gradient  dtable = scale P^T dy           (sums over the tokens of each row)
// The gradient takes the ids sorted by value (a route with k = 1 over V keys),
// so every table row is written once, by one CTA, with its tokens added in a
// fixed order: no atomics on values, the same bits on every run.  A frequent
// token would leave its row to one CTA for long, so sums of whole chunks of 32
// sorted tokens that lie inside one row's run are formed first, in parallel, and
// sums of 32 such chunks in a second step; the row's CTA adds at most 31 tokens,
// 31 chunks and the groups on each side.  Both kernels are bound by HBM: the
// gradient by writing V rows.
#include "internal.h"
#include "rowvec.cuh"
#include "sm103.cuh"

namespace spmm {
namespace {

using namespace rows;

constexpr int kRowThreads = 256;
constexpr int kFlight = 8;   // rows in flight per thread while summing
constexpr int kChunk = 32;   // sorted tokens per partial sum, and partial sums per group

struct EmbedArgs {
    const void* table;
    int64_t ldt, V, H;
    const void* ids;
    int32_t wide;
    float scale;
    void* out;
    int64_t ldo;
    int* err;
};

// One CTA per token.
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) embed_kernel(const EmbedArgs a) {
    using X = Vec<T, V>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t t = blockIdx.x;
    const int64_t id =
        a.wide ? __ldg(static_cast<const int64_t*>(a.ids) + t) : __ldg(static_cast<const int32_t*>(a.ids) + t);
    const bool live = id >= 0 && id < a.V;
    if (id >= a.V && threadIdx.x == 0) atomicOr(a.err, SPMM_DEVERR_INDEX);
    const T* row = static_cast<const T*>(a.table) + (live ? id : 0) * a.ldt;
    T* out = static_cast<T*>(a.out) + t * a.ldo;
    for (int64_t c = threadIdx.x * V; c < a.H; c += 2 * blockDim.x * V) {
        const int64_t c1 = c + blockDim.x * V;
        const bool two = c1 < a.H;
        const typename X::Raw r0 = live ? X::load(row + c) : X::zero(), r1 = live && two ? X::load(row + c1) : X::zero();
        float f[V];
        X::unpack(r0, f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= live ? a.scale : 1.f;
        X::store(out + c, X::pack(f));
        if (!two) break;
        X::unpack(r1, f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= live ? a.scale : 1.f;
        X::store(out + c1, X::pack(f));
    }
}

struct EmbedGradArgs {
    const int32_t *order, *offsets;
    int64_t T, V, H;
    const void* dy;
    int64_t ldy;
    float scale;
    bool accumulate;
    void* out;
    int64_t ldo;
    float *chunks, *groups;  // [T / 32][Hp], [T / 1024][Hp]
    int64_t Hp;
};

// acc += rows at(0) .. at(n - 1) of p, in order.
template <typename T, int V, typename At>
__device__ __forceinline__ void add_rows(const T* p, int n, At at, float (&acc)[V]) {
    using X = Vec<T, V>;
    for (int i0 = 0; i0 < n; i0 += kFlight) {
        typename X::Raw r[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) r[i] = i0 + i < n ? X::load(p + at(i0 + i)) : X::zero();
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            float f[V];
            X::unpack(r[i], f);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += f[k];
        }
    }
}

// The row whose run holds sorted place p: the last v with offsets[v] <= p, by a
// 32-way search of one warp.
__device__ __forceinline__ int64_t row_of(const int32_t* offsets, int64_t V, int64_t p, int lane) {
    int64_t lo = 0, hi = V;  // offsets[lo] <= p < offsets[hi]
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + step * lane;
        const uint32_t le = __ballot_sync(0xffffffffu, at < hi && __ldg(offsets + at) <= p);
        lo += step * (31 - __clz(le));
        hi = lo + step < hi ? lo + step : hi;
    }
    return lo;
}

// Sums of whole chunks (LEVEL 0: of tokens, LEVEL 1: of chunks) inside one run.
// Grid (units, column pieces).
template <typename T, int V, int LEVEL>
__global__ void __launch_bounds__(kRowThreads) embed_partial_kernel(const EmbedGradArgs a) {
    constexpr int64_t kSpan = LEVEL ? kChunk * kChunk : kChunk;
    __shared__ int32_t row[kChunk];
    __shared__ int whole;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t p0 = blockIdx.x * kSpan;
    if (threadIdx.x < 32) {
        bool inside = p0 + kSpan <= __ldg(a.offsets + a.V);
        if (inside) inside = __ldg(a.offsets + row_of(a.offsets, a.V, p0, threadIdx.x) + 1) >= p0 + kSpan;
        if (threadIdx.x == 0) whole = inside;
        if (!LEVEL && inside) row[threadIdx.x] = __ldg(a.order + p0 + threadIdx.x);
    }
    __syncthreads();
    if (!whole) return;
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * V;
    if (c >= a.H) return;
    float acc[V] = {};
    if (LEVEL) {
        const float* src = a.chunks + blockIdx.x * kChunk * a.Hp + c;
        add_rows<float, V>(src, kChunk, [&](int i) { return i * a.Hp; }, acc);
        Vec<float, V>::store(a.groups + blockIdx.x * a.Hp + c, Vec<float, V>::pack(acc));
    } else {
        add_rows<T, V>(static_cast<const T*>(a.dy) + c, kChunk, [&](int i) { return row[i] * a.ldy; }, acc);
        Vec<float, V>::store(a.chunks + blockIdx.x * a.Hp + c, Vec<float, V>::pack(acc));
    }
}

// kRows table rows per CTA.
constexpr int kRows = 4;

template <typename T, int V, typename TO>
__global__ void __launch_bounds__(kRowThreads) embed_grad_kernel(const EmbedGradArgs a) {
    using O = Vec<TO, V>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kRows;
    int32_t start[kRows + 1];
#pragma unroll
    for (int i = 0; i <= kRows; ++i) start[i] = __ldg(a.offsets + (v0 + i < a.V ? v0 + i : a.V));
    const T* dy = static_cast<const T*>(a.dy);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int32_t p0 = start[i], p1 = start[i + 1];
        if (v0 + i >= a.V) return;
        TO* out = static_cast<TO*>(a.out) + (v0 + i) * a.ldo;
        if (p0 == p1) {
            if (!a.accumulate)
                for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) O::store_cs(out + c, O::zero());
            continue;
        }
        // tokens up to the first whole chunk, chunks up to the first whole group, groups, and back
        const int32_t c0 = (p0 + kChunk - 1) / kChunk, c1 = max(c0, p1 / kChunk);
        const bool chunked = c0 < c1;
        const int32_t g0 = (c0 + kChunk - 1) / kChunk, g1 = max(g0, c1 / kChunk);
        const bool grouped = g0 < g1;
        const int32_t t_end = chunked ? c0 * kChunk : p1, c_end = grouped ? g0 * kChunk : c1;
        for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) {
            float acc[V] = {};
            const auto token = [&](int32_t p) { return static_cast<int64_t>(__ldg(a.order + p)) * a.ldy; };
            add_rows<T, V>(dy + c, t_end - p0, [&](int k) { return token(p0 + k); }, acc);
            if (chunked) {
                add_rows<float, V>(a.chunks + c, c_end - c0, [&](int k) { return (c0 + k) * a.Hp; }, acc);
                if (grouped) {
                    add_rows<float, V>(a.groups + c, g1 - g0, [&](int k) { return (g0 + k) * a.Hp; }, acc);
                    add_rows<float, V>(a.chunks + c, c1 - g1 * kChunk, [&](int k) { return (g1 * kChunk + k) * a.Hp; },
                                       acc);
                }
                add_rows<T, V>(dy + c, p1 - c1 * kChunk, [&](int k) { return token(c1 * kChunk + k); }, acc);
            }
            float base[V] = {};
            if (a.accumulate) O::unpack(*reinterpret_cast<const typename O::Raw*>(out + c), base);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = fmaf(a.scale, acc[k], base[k]);
            O::store_cs(out + c, O::pack(acc));
        }
    }
}

int64_t padded(int64_t H) { return (H + 7) / 8 * 8; }

template <typename T, int V, typename TO>
cudaError_t embed_grad(const EmbedGradArgs& a, cudaStream_t s) {
    const int threads = row_threads(a.H, V, kRowThreads);
    const unsigned pieces = static_cast<unsigned>((a.H + threads * V - 1) / (threads * V));
    cudaError_t e = cudaSuccess;
    if (a.T >= kChunk)
        e = launch_chained(embed_partial_kernel<T, V, 0>, dim3(static_cast<unsigned>(a.T / kChunk), pieces), threads, 0, 1,
                           s, a);
    if (a.T >= kChunk * kChunk && e == cudaSuccess)
        e = launch_chained(embed_partial_kernel<T, V, 1>, dim3(static_cast<unsigned>(a.T / (kChunk * kChunk)), pieces),
                           threads, 0, 1, s, a);
    if (e != cudaSuccess) return e;
    return launch_chained(embed_grad_kernel<T, V, TO>, static_cast<unsigned>((a.V + kRows - 1) / kRows), threads, 0, 1, s,
                          a);
}

template <typename T, int V>
cudaError_t embed_grad_to(const EmbedGradArgs& a, bool f32, cudaStream_t s) {
    return f32 ? embed_grad<T, V, float>(a, s) : embed_grad<T, V, T>(a, s);
}

}  // namespace

spmm_status launch_embed(const void* table, int64_t V, int64_t H, int64_t ldt, int32_t dtype, const void* ids,
                         int32_t id_bytes, int64_t T, float scale, void* out, int64_t ldo, cudaStream_t s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return SPMM_ERR_CUDA;
    EmbedArgs a{table, ldt, V, H, ids, id_bytes == 8, scale, out, ldo, dev->err};
    const int es = row_elem_bytes(dtype);
    const bool v = rows16(table, ldt, H, es) && rows16(out, ldo, H, es);
    const unsigned grid = static_cast<unsigned>(T);
    const int threads = row_threads(H, v ? 16 / es : 1, kRowThreads);
    cudaError_t e;
    trace_begin(SPMM_KERNEL_ROWS, s);
    SPMM_ROWS_TYPED(e, dtype, v, embed_kernel, grid, threads, s, a);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(e);
}

size_t embed_grad_workspace_bytes(int64_t T, int64_t H) {
    return static_cast<size_t>(T / kChunk + T / (kChunk * kChunk)) * padded(H) * sizeof(float);
}

spmm_status launch_embed_grad(const spmm_route_t* R, const void* dy, int64_t ldy, int64_t H, int32_t dtype, float scale,
                              bool accumulate, void* out, int64_t ldo, int32_t out_dtype, void* ws, cudaStream_t s) {
    EmbedGradArgs a{};
    a.order = R->order;
    a.offsets = R->offsets;
    a.T = R->T;
    a.V = R->n_keys;
    a.H = H;
    a.dy = dy;
    a.ldy = ldy;
    a.scale = scale;
    a.accumulate = accumulate;
    a.out = out;
    a.ldo = ldo;
    a.Hp = padded(H);
    a.chunks = static_cast<float*>(ws);
    a.groups = a.chunks + R->T / kChunk * a.Hp;
    const bool v = rows16(dy, ldy, H, row_elem_bytes(dtype)) && rows16(out, ldo, H, row_elem_bytes(out_dtype));
    const bool f32 = out_dtype == SPMM_F32;
    cudaError_t e;
    trace_begin(SPMM_KERNEL_ROWS, s);
    if (dtype == SPMM_F32)
        e = v ? embed_grad<float, 4, float>(a, s) : embed_grad<float, 1, float>(a, s);
    else if (dtype == SPMM_F16)
        e = v ? embed_grad_to<__half, 8>(a, f32, s) : embed_grad_to<__half, 1>(a, f32, s);
    else
        e = v ? embed_grad_to<__nv_bfloat16, 8>(a, f32, s) : embed_grad_to<__nv_bfloat16, 1>(a, f32, s);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(e);
}

}  // namespace spmm
