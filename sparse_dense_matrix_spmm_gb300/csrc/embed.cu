// embed.cu -- embedding lookup and its gradient: products with the T x V one-hot
// matrix of token ids.
//   lookup    out    = scale P table          (out[t] = scale table[ids[t]])
//   gradient  dtable = scale P^T dy           (sums over the tokens of each row)
// The gradient takes the ids sorted by value (a route with k = 1 over V keys) and
// reads every row of dy once: a CTA adds up 64 consecutive sorted tokens, writes
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
constexpr int kFlightWide = 8;    // rows in flight per thread while summing,
constexpr int kFlightNarrow = 4;  // and in moves below 8 bytes (8 rows: 5% slower)
constexpr int kJoin = 8;     // partial sums in flight per thread
constexpr int kChunk = 64;   // sorted tokens per CTA (32: twice the partial sums, 4 us more at 32768 tokens)
constexpr int kSumThreads = 256;
constexpr int kZeroRows = 4; // table rows per CTA that zeroes
constexpr int kBoundaries = 2;  // chunk boundaries per CTA that joins

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
    using X = Cols<T, V, 2, 2>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t t = blockIdx.x;
    const int64_t id =
        a.wide ? static_cast<const int64_t*>(a.ids)[t] : static_cast<const int32_t*>(a.ids)[t];
    const bool live = id >= 0 && id < a.V;
    if (id >= a.V && threadIdx.x == 0) atomicOr(a.err, SPMM_DEVERR_INDEX);
    const T* row = static_cast<const T*>(a.table) + (live ? id : 0) * a.ldt;
    T* out = static_cast<T*>(a.out) + t * a.ldo;
    const float scale = live ? a.scale : 1.f;
    const int step = blockDim.x * V;
    for (int64_t c = threadIdx.x * V; c < a.H; c += X::U * step) {
        typename X::Raw r[X::U];
        if (live)
            X::load(r, row, c, a.H, step);
        else
            X::clear(r);
        float f[X::N];
        X::unpack(r, f);
#pragma unroll
        for (int i = 0; i < X::N; ++i) f[i] *= scale;
        X::pack(r, f);
        X::store_cs(out, r, c, a.H, step);
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
    if (a.accumulate) O::unpack(O::load(out), f);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = fmaf(a.scale, acc[k], f[k]);
    O::store_cs(out, O::pack(f));
}

// Blocks [0, chunks x pieces): sums of a chunk's tokens over a piece of the
// columns.  The blocks after them zero rows without tokens.
template <typename T, int V, typename TO>
__global__ void __launch_bounds__(kSumThreads) embed_grad_kernel(const EmbedGradArgs a, int pieces) {
    using X = Vec<T, V>;
    using O = Vec<TO, V>;
    using F = Vec<float, V>;
    constexpr int kFlight = V * sizeof(T) < 8 ? kFlightNarrow : kFlightWide;
    __shared__ int32_t token[kChunk], key[kChunk + 2];  // key[i + 1] of token i; neighbours at the ends
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t block = blockIdx.x;
    if (block >= a.chunks * pieces) {
        const int64_t v0 = (block - a.chunks * pieces) * kZeroRows;
        int32_t start[kZeroRows + 1];
#pragma unroll
        for (int i = 0; i <= kZeroRows; ++i) start[i] = a.offsets[v0 + i < a.V ? v0 + i : a.V];
#pragma unroll
        for (int i = 0; i < kZeroRows; ++i) {
            if (v0 + i >= a.V || start[i] != start[i + 1]) continue;
            TO* out = static_cast<TO*>(a.out) + (v0 + i) * a.ldo;
            for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) O::store_cs(out + c, O::zero());
        }
        return;
    }
    const int64_t chunk = block / pieces, p0 = chunk * kChunk;
    const int64_t kept = a.offsets[a.V];
    if (p0 >= kept) return;
    const int n = static_cast<int>(kept - p0 < kChunk ? kept - p0 : kChunk);
    for (int i = threadIdx.x; i < kChunk + 2; i += blockDim.x) {
        const int64_t p = p0 + i - 1;
        const bool in = p >= 0 && p < kept;
        key[i] = in ? a.keys[p] : -1;
        if (i >= 1 && i <= kChunk) token[i - 1] = in ? a.order[p] : 0;
    }
    __syncthreads();
    const int64_t c = ((block - chunk * pieces) * blockDim.x + threadIdx.x) * V;
    if (c >= a.H) return;
    const T* dy = static_cast<const T*>(a.dy) + c;
    bool entered = key[0] == key[1];  // the current run began in an earlier chunk
    float acc[V] = {};
    for (int i0 = 0; i0 < n; i0 += kFlight) {
        typename X::Raw r[kFlight];
        if (i0 + kFlight <= n) {  // loads without a test each: 4095 columns 139 us, with 144
#pragma unroll
            for (int i = 0; i < kFlight; ++i) r[i] = X::load_cs(dy + token[i0 + i] * a.ldy);
        } else {
#pragma unroll
            for (int i = 0; i < kFlight; ++i) r[i] = i0 + i < n ? X::load_cs(dy + token[i0 + i] * a.ldy) : X::zero();
        }
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
                F::store(a.partial + (2 * chunk + (entered ? 0 : 1)) * a.Hp + c, F::pack(acc));
            else
                write_row<V, TO>(a, v, c, acc);
            entered = false;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
        }
    }
}

// acc += partial sums q0 .. q1 - 1 of a run at column c: number 0 is the tail of
// the chunk it began in, number q > 0 the head of chunk first + q - 1.
template <int V>
__device__ __forceinline__ void add_partial(const EmbedGradArgs& a, int64_t first, int64_t q0, int64_t q1, int64_t c,
                                            float (&acc)[V]) {
    using F = Vec<float, V>;
    const float* src = a.partial + (2 * first - 2) * a.Hp + c;
    for (int64_t q = q0; q < q1; q += kJoin) {
        typename F::Raw r[kJoin];
#pragma unroll
        for (int k = 0; k < kJoin; ++k)
            r[k] = q + k < q1 ? F::load(src + (q + k ? 2 * (q + k) : 1) * a.Hp) : F::zero();
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            float f[V];
            F::unpack(r[k], f);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += f[j];
        }
    }
}

// Block (group of boundaries, piece of the columns): the runs that cross into a
// chunk from the chunk they began in, for kBoundaries chunks.  Most boundaries
// start no such run (a frequent token's run crosses many but starts once), so
// one thread each looks at them first.  A short run is added by each thread for
// its columns; the partial sums of a long one are shared out over the warps in
// consecutive parts, and the parts added in order.  dy is read with evict-first
// loads so that the partial sums are still in L2 here: 32768 tokens on one row
// take 95 us in all, 245 us with plain loads and 32 tokens per chunk.
template <int V, typename TO>
__global__ void __launch_bounds__(kRowThreads) embed_join_kernel(const EmbedGradArgs a) {
    constexpr int kWarps = kRowThreads / 32;
    __shared__ int32_t row[kBoundaries], last[kBoundaries];  // row -1: nothing to join
    __shared__ float part[kWarps][kRowThreads * V];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kBoundaries + 1;  // chunk of the first boundary
    if (threadIdx.x < kBoundaries) {
        const int64_t p = (first + threadIdx.x) * kChunk;
        int32_t v = -1, end = 0;
        if (p < a.T) {
            const int32_t here = a.keys[p], before = a.keys[p - 1];
            if (here == before && here < a.V && a.offsets[here] >= p - kChunk) {
                v = here;
                end = a.offsets[here + 1];
            }
        }
        row[threadIdx.x] = v;
        last[threadIdx.x] = (end - 1) / kChunk;
    }
    __syncthreads();
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kRowThreads * V, c = c0 + threadIdx.x * V;
    for (int i = 0; i < kBoundaries; ++i) {
        const int32_t v = row[i];
        if (v < 0) continue;
        const int64_t n = last[i] - (first + i) + 2;
        float acc[V] = {};
        if (n <= 2 * kJoin) {
            if (c >= a.H) continue;
            add_partial<V>(a, first + i, 0, n, c, acc);
        } else {
            const int64_t per = (n + kWarps - 1) / kWarps, q0 = warp * per, q1 = q0 + per < n ? q0 + per : n;
            for (int s = 0; s < kWarps; ++s) {  // this warp's part, 32 V columns at a time
                const int at = (s * 32 + lane) * V;
                float f[V] = {};
                if (c0 + at < a.H) add_partial<V>(a, first + i, q0, q1, c0 + at, f);
#pragma unroll
                for (int j = 0; j < V; ++j) part[warp][at + j] = f[j];
            }
            __syncthreads();
            for (int w = 0; w < kWarps; ++w)
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] += part[w][threadIdx.x * V + j];
            __syncthreads();
            if (c >= a.H) continue;
        }
        write_row<V, TO>(a, v, c, acc);
    }
}

int64_t padded(int64_t H) { return (H + 7) / 8 * 8; }

template <typename T, int V, typename TO>
cudaError_t embed_grad(const EmbedGradArgs& a, cudaStream_t s) {
    const int threads = row_threads(a.H, V, kSumThreads);
    const int64_t pieces = (a.H + threads * V - 1) / (threads * V);
    const int64_t zeros = a.accumulate ? 0 : (a.V + kZeroRows - 1) / kZeroRows;
    const int64_t blocks = a.chunks * pieces + zeros;
    if (blocks == 0) return cudaSuccess;
    if (blocks >= (int64_t(1) << 31)) return cudaErrorNotSupported;
    cudaError_t e = launch_chained(embed_grad_kernel<T, V, TO>, static_cast<unsigned>(blocks), threads, 0, 1, s, a,
                                   static_cast<int>(pieces));
    if (e != cudaSuccess || a.chunks < 2) return e;
    constexpr int VJ = V > 4 ? 4 : V;  // 16 bytes of a partial sum
    constexpr int64_t kAcross = 65535, kSpan = kRowThreads * VJ;  // a grid's rows; columns of a piece
    for (int64_t c = 0; c < a.H && e == cudaSuccess; c += kAcross * kSpan) {
        EmbedGradArgs b = a;
        b.H = a.H - c;
        b.out = static_cast<TO*>(a.out) + c;
        b.partial = a.partial + c;
        if (b.H > kAcross * kSpan) b.H = kAcross * kSpan;
        const dim3 grid(static_cast<unsigned>((a.chunks - 1 + kBoundaries - 1) / kBoundaries),
                        static_cast<unsigned>((b.H + kSpan - 1) / kSpan));
        e = launch_chained(embed_join_kernel<VJ, TO>, grid, kRowThreads, 0, 1, s, b);
    }
    return e;
}

template <typename T, int V>
cudaError_t embed_grad_to(const EmbedGradArgs& a, bool f32, cudaStream_t s) {
    return f32 ? embed_grad<T, V, float>(a, s) : embed_grad<T, V, T>(a, s);
}

template <typename T>
cudaError_t embed_grad_16(const EmbedGradArgs& a, int v, bool f32, cudaStream_t s) {
    return v == 8   ? embed_grad_to<T, 8>(a, f32, s)
           : v == 4 ? embed_grad_to<T, 4>(a, f32, s)
           : v == 2 ? embed_grad_to<T, 2>(a, f32, s)
                    : embed_grad_to<T, 1>(a, f32, s);
}

}  // namespace

spmm_status launch_embed(const void* table, int64_t V, int64_t H, int64_t ldt, int32_t dtype, const void* ids,
                         int32_t id_bytes, int64_t T, float scale, void* out, int64_t ldo, cudaStream_t s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return SPMM_ERR_CUDA;
    EmbedArgs a{table, ldt, V, H, ids, id_bytes == 8, scale, out, ldo, dev->err};
    const int es = row_elem_bytes(dtype);
    const Operand o[] = {{table, ldt, es}, {out, ldo, es}};
    const int v = row_width(o, H);
    const unsigned grid = static_cast<unsigned>(T);
    const int threads = row_threads(H, 16 / es, kRowThreads);
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
    const Operand o[] = {{dy, ldy, row_elem_bytes(dtype)}, {out, ldo, row_elem_bytes(out_dtype)}};
    const int v = row_width(o, H);
    const bool f32 = out_dtype == SPMM_F32;
    cudaError_t e;
    trace_begin(SPMM_KERNEL_ROWS, s);
    if (dtype == SPMM_F32)
        e = v == 4   ? embed_grad<float, 4, float>(a, s)
            : v == 2 ? embed_grad<float, 2, float>(a, s)
                     : embed_grad<float, 1, float>(a, s);
    else if (dtype == SPMM_F16)
        e = embed_grad_16<__half>(a, v, f32, s);
    else
        e = embed_grad_16<__nv_bfloat16>(a, v, f32, s);
    trace_end(SPMM_KERNEL_ROWS, s);
    return e == cudaErrorNotSupported ? SPMM_ERR_UNSUPPORTED : cuda_status(e);  // a grid of 2^31 CTAs or more
}

}  // namespace spmm
