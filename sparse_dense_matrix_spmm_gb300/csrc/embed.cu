// embed.cu -- embedding lookup and its gradient: products with the T x V one-hot
// matrix of token ids.
//   lookup    out    = scale P table          (out[t] = scale table[ids[t]])
//   gradient  dtable = scale P^T dy           (sums over the tokens of each row)
// The gradient takes the ids sorted by value (a route with k = 1 over V keys),
// so every table row is written once, by one CTA, with its tokens added in
// input order: no atomics on values, the same bits on every run.
#include "internal.h"
#include "rowvec.cuh"

namespace spmm {
namespace {

using namespace rows;

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
__global__ void embed_kernel(const EmbedArgs a) {
    using X = Vec<T, V>;
    const int64_t t = blockIdx.x;
    const int64_t id = a.wide ? static_cast<const int64_t*>(a.ids)[t] : static_cast<const int32_t*>(a.ids)[t];
    const bool live = id >= 0 && id < a.V;
    if (id >= a.V && threadIdx.x == 0) atomicOr(a.err, SPMM_DEVERR_INDEX);
    const T* row = static_cast<const T*>(a.table) + (live ? id : 0) * a.ldt;
    T* out = static_cast<T*>(a.out) + t * a.ldo;
    for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) {
        float f[V] = {};
        if (live) {
            X::unpack(X::load(row + c), f);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= a.scale;
        }
        X::store(out + c, X::pack(f));
    }
}

struct EmbedGradArgs {
    const int32_t *order, *offsets;
    int64_t V, H;
    const void* dy;
    int64_t ldy;
    float scale;
    bool accumulate;
    void* out;
    int64_t ldo;
};

// One CTA per table row.
template <typename T, int V, typename TO>
__global__ void embed_grad_kernel(const EmbedGradArgs a) {
    using X = Vec<T, V>;
    using O = Vec<TO, V>;
    const int64_t v = blockIdx.x;
    const int32_t p0 = a.offsets[v], p1 = a.offsets[v + 1];
    if (a.accumulate && p0 == p1) return;
    const T* dy = static_cast<const T*>(a.dy);
    TO* out = static_cast<TO*>(a.out) + v * a.ldo;
    for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) {
        float acc[V] = {};
        for (int32_t p = p0; p < p1; ++p) {
            float f[V];
            X::unpack(X::load(dy + a.order[p] * a.ldy + c), f);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += f[i];
        }
        float base[V] = {};
        if (a.accumulate) O::unpack(*reinterpret_cast<const typename O::Raw*>(out + c), base);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(a.scale, acc[i], base[i]);
        O::store(out + c, O::pack(acc));
    }
}

int row_threads(int64_t H, int v) {
    const int64_t n = (H + v - 1) / v;
    return n >= 512 ? 512 : static_cast<int>((n + 31) / 32 * 32);
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
    const int threads = row_threads(H, v ? 16 / es : 1);
    trace_begin(SPMM_KERNEL_ROWS, s);
    SPMM_ROWS_TYPED(dtype, v, embed_kernel, grid, threads, s, a);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(cudaGetLastError());
}

size_t embed_grad_workspace_bytes(int64_t, int64_t) { return 0; }

spmm_status launch_embed_grad(const spmm_route_t* R, const void* dy, int64_t ldy, int64_t H, int32_t dtype, float scale,
                              bool accumulate, void* out, int64_t ldo, int32_t out_dtype, void*, cudaStream_t s) {
    const EmbedGradArgs a{R->order, R->offsets, R->n_keys, H, dy, ldy, scale, accumulate, out, ldo};
    const bool v = rows16(dy, ldy, H, row_elem_bytes(dtype)) && rows16(out, ldo, H, row_elem_bytes(out_dtype));
    const unsigned grid = static_cast<unsigned>(R->n_keys);
    const int threads = row_threads(H, v ? 16 / row_elem_bytes(dtype) : 1);
    trace_begin(SPMM_KERNEL_ROWS, s);
    if (dtype == SPMM_F32)
        v ? embed_grad_kernel<float, 4, float><<<grid, threads, 0, s>>>(a)
          : embed_grad_kernel<float, 1, float><<<grid, threads, 0, s>>>(a);
    else if (dtype == SPMM_F16)
        out_dtype == SPMM_F32 ? (v ? embed_grad_kernel<__half, 8, float><<<grid, threads, 0, s>>>(a)
                                   : embed_grad_kernel<__half, 1, float><<<grid, threads, 0, s>>>(a))
                              : (v ? embed_grad_kernel<__half, 8, __half><<<grid, threads, 0, s>>>(a)
                                   : embed_grad_kernel<__half, 1, __half><<<grid, threads, 0, s>>>(a));
    else
        out_dtype == SPMM_F32
            ? (v ? embed_grad_kernel<__nv_bfloat16, 8, float><<<grid, threads, 0, s>>>(a)
                 : embed_grad_kernel<__nv_bfloat16, 1, float><<<grid, threads, 0, s>>>(a))
            : (v ? embed_grad_kernel<__nv_bfloat16, 8, __nv_bfloat16><<<grid, threads, 0, s>>>(a)
                 : embed_grad_kernel<__nv_bfloat16, 1, __nv_bfloat16><<<grid, threads, 0, s>>>(a));
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(cudaGetLastError());
}

}  // namespace spmm
