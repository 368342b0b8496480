// embed.cu -- embedding lookup and its gradient: products with the T x V one-hot
// matrix of token ids.
//   lookup    out    = scale P table          (out[t] = scale table[ids[t]])
//   gradient  dtable = scale P^T dy           (sums over the tokens of each row)
// The gradient takes the ids sorted by value (a route with k = 1 over V keys) and
// reads every row of dy once: a CTA adds up 32 consecutive sorted tokens, writes
// the rows whose tokens all lie among them, and leaves a partial sum at either
// end; a second launch joins the partial sums of rows that cross a boundary.  So
// a frequent token is as parallel as rare ones (one CTA per table row left a row
// of 1700 tokens to one CTA, 0.7 ms), nothing is added with atomics, and the
// result has the same bits on every run.  Rows without tokens are zeroed by the
// first launch's other CTAs, in address order beside the sums: the operator is
// bound by writing V rows to HBM.
#include "internal.h"
#include "rowvec.cuh"
#include "sm103_more.cuh"

namespace spmm {
namespace {

using namespace rows;

constexpr int kRowThreads = 256;
constexpr int kFlight = 8;   // rows in flight per thread while summing
constexpr int kJoin = 16;    // partial sums in flight per thread
constexpr int kChunk = 32;   // sorted tokens per CTA
constexpr int kZeroRows = 4; // table rows per CTA that zeroes

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
    const int32_t *order, *keys, *offsets;
    int64_t T, V, H, chunks;
    const void* dy;
    int64_t ldy;
    float scale;
    bool accumulate;
    void* out;
    int64_t ldo;
    float* partial;  // [chunks][2][Hp]: the run that entered the chunk, the run that leaves it
    int64_t Hp;
};

// out = base + scale acc, the base only when accumulating.
template <int V, typename TO>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, int64_t v, int64_t c, const float (&acc)[V]) {
    using O = Vec<TO, V>;
    TO* out = static_cast<TO*>(a.out) + v * a.ldo + c;
    float f[V] = {};
    if (a.accumulate) O::unpack(*reinterpret_cast<const typename O::Raw*>(out), f);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = fmaf(a.scale, acc[k], f[k]);
    O::store_cs(out, O::pack(f));
}

// Blocks [0, chunks x pieces): sums of a chunk's tokens over a piece of the
// columns.  The blocks after them zero rows without tokens.
template <typename T, int V, typename TO>
__global__ void __launch_bounds__(kRowThreads) embed_grad_kernel(const EmbedGradArgs a, int pieces) {
    using X = Vec<T, V>;
    using O = Vec<TO, V>;
    __shared__ int32_t token[kChunk], key[kChunk + 2];  // key[i + 1] of token i; neighbours at the ends
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t block = blockIdx.x;
    if (block >= a.chunks * pieces) {
        const int64_t v0 = (block - a.chunks * pieces) * kZeroRows;
        int32_t start[kZeroRows + 1];
#pragma unroll
        for (int i = 0; i <= kZeroRows; ++i) start[i] = __ldg(a.offsets + (v0 + i < a.V ? v0 + i : a.V));
#pragma unroll
        for (int i = 0; i < kZeroRows; ++i) {
            if (v0 + i >= a.V || start[i] != start[i + 1]) continue;
            TO* out = static_cast<TO*>(a.out) + (v0 + i) * a.ldo;
            for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) O::store_cs(out + c, O::zero());
        }
        return;
    }
    const int64_t chunk = block / pieces, p0 = chunk * kChunk;
    const int64_t kept = __ldg(a.offsets + a.V);
    if (p0 >= kept) return;
    const int n = static_cast<int>(kept - p0 < kChunk ? kept - p0 : kChunk);
    if (threadIdx.x < 32) {
        const int64_t p = p0 + threadIdx.x;
        token[threadIdx.x] = p < kept ? __ldg(a.order + p) : 0;
        key[threadIdx.x + 1] = p < kept ? __ldg(a.keys + p) : -1;
        if (threadIdx.x == 0) {
            key[0] = p0 > 0 ? __ldg(a.keys + p0 - 1) : -1;
            key[kChunk + 1] = p0 + kChunk < kept ? __ldg(a.keys + p0 + kChunk) : -1;
        }
    }
    __syncthreads();
    const int64_t c = ((block - chunk * pieces) * blockDim.x + threadIdx.x) * V;
    if (c >= a.H) return;
    const T* dy = static_cast<const T*>(a.dy) + c;
    bool entered = key[0] == key[1];  // the current run began in an earlier chunk
    float acc[V] = {};
    for (int i0 = 0; i0 < n; i0 += kFlight) {
        typename X::Raw r[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) r[i] = i0 + i < n ? X::load(dy + token[i0 + i] * a.ldy) : X::zero();
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            if (i0 + i >= n) break;
            float f[V];
            X::unpack(r[i], f);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += f[k];
            const int32_t v = key[i0 + i + 1];
            const bool leaves = i0 + i + 1 == n && key[n + 1] == v;
            if (!leaves && key[i0 + i + 2] == v) continue;
            if (entered || leaves)
                Vec<float, V>::store(a.partial + (2 * chunk + (entered ? 0 : 1)) * a.Hp + c, Vec<float, V>::pack(acc));
            else
                write_row<V, TO>(a, v, c, acc);
            entered = false;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
        }
    }
}

// Block (chunk - 1, piece): the run that crosses into `chunk` from the chunk it
// began in.
template <int V, typename TO>
__global__ void __launch_bounds__(kRowThreads) embed_join_kernel(const EmbedGradArgs a) {
    using F = Vec<float, V>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t chunk = static_cast<int64_t>(blockIdx.x) + 1, p = chunk * kChunk;
    if (p >= __ldg(a.offsets + a.V)) return;
    const int32_t v = __ldg(a.keys + p);
    if (__ldg(a.keys + p - 1) != v || __ldg(a.offsets + v) < p - kChunk) return;
    const int64_t last = (__ldg(a.offsets + v + 1) - 1) / kChunk;
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * V;
    if (c >= a.H) return;
    float acc[V];
    F::unpack(F::load(a.partial + (2 * chunk - 1) * a.Hp + c), acc);
    for (int64_t q = chunk; q <= last; q += kJoin) {
        typename F::Raw r[kJoin];
#pragma unroll
        for (int i = 0; i < kJoin; ++i) r[i] = q + i <= last ? F::load(a.partial + 2 * (q + i) * a.Hp + c) : F::zero();
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            float f[V];
            F::unpack(r[i], f);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += f[k];
        }
    }
    write_row<V, TO>(a, v, c, acc);
}

int64_t padded(int64_t H) { return (H + 7) / 8 * 8; }

template <typename T, int V, typename TO>
cudaError_t embed_grad(const EmbedGradArgs& a, cudaStream_t s) {
    const int threads = row_threads(a.H, V, kRowThreads);
    const int64_t pieces = (a.H + threads * V - 1) / (threads * V);
    const int64_t zeros = a.accumulate ? 0 : (a.V + kZeroRows - 1) / kZeroRows;
    const int64_t blocks = a.chunks * pieces + zeros;
    if (blocks == 0) return cudaSuccess;
    if (blocks >= (int64_t(1) << 31) || pieces >= 65536) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_chained(embed_grad_kernel<T, V, TO>, static_cast<unsigned>(blocks), threads, 0, 1, s, a,
                                         static_cast<int>(pieces));
    if (e != cudaSuccess || a.chunks < 2) return e;
    constexpr int VJ = V > 4 ? 4 : V;  // 16 bytes of a partial sum
    const int jthreads = row_threads(a.H, VJ, kRowThreads);
    const dim3 grid(static_cast<unsigned>(a.chunks - 1), static_cast<unsigned>((a.H + jthreads * VJ - 1) / (jthreads * VJ)));
    return launch_chained(embed_join_kernel<VJ, TO>, grid, jthreads, 0, 1, s, a);
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
    return static_cast<size_t>((T + kChunk - 1) / kChunk) * 2 * padded(H) * sizeof(float);
}

spmm_status launch_embed_grad(const spmm_route_t* R, const void* dy, int64_t ldy, int64_t H, int32_t dtype, float scale,
                              bool accumulate, void* out, int64_t ldo, int32_t out_dtype, void* ws, cudaStream_t s) {
    EmbedGradArgs a{};
    a.order = R->order;
    a.keys = R->keys;
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
    a.chunks = (R->T + kChunk - 1) / kChunk;
    a.partial = static_cast<float*>(ws);
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
