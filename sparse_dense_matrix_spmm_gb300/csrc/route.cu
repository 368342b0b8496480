// route.cu -- one-hot sparse matrices stored by their sorted rows, and the
// products with them that move rows.
//
// A route is the stable sort of R = T k integers ids[t][j] by value: order[p]
// is the flat index f = t k + j at place p, pos[f] its place, offsets[e] the
// first place of key e.  With P the R x T matrix P[p][order[p] / k] = 1:
//   dispatch       xs  = P x
//   combine        y   = P^T diag(w) ys      (w in sorted order)
//   combine grad   dys = diag(w) P dy,  dw[p] = <ys[p], (P dy)[p]>
// All three move each row once and are bound by HBM.
#include "internal.h"
#include "rowvec.cuh"
#include "sm103.cuh"

namespace spmm {
namespace {

using namespace rows;

// ---------------------------------------------------------------- sort
// Least-significant-digit radix sort with 9-bit digits in one CTA.  Every warp
// owns a consecutive piece of the input, so "earlier warp, then earlier lane" is
// input order and each pass is stable.  A pass counts digits per warp, turns the
// counts into first places (digits, then warps, in order) and writes each
// element at its digit's next place in its warp.
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortWarps = 32;

struct SortArgs {
    const void* ids;
    int64_t ldi;      // row pitch of ids in elements
    int32_t wide;     // ids are 64-bit
    int32_t k, n, n_keys, passes;
    int32_t *order, *pos, *offsets;
    int32_t *key_buf[2], *idx_buf[2];  // between passes
    int* err;
};

// Key of flat index f: its id, or n_keys (sorted last) when the choice is dropped.
__device__ __forceinline__ int32_t load_key(const SortArgs& a, int32_t f) {
    const int32_t t = f / a.k;
    const int64_t at = t * a.ldi + (f - t * a.k);
    const int64_t v = a.wide ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
    if (v >= 0 && v < a.n_keys) return static_cast<int32_t>(v);
    if (v >= 0) atomicOr(a.err, SPMM_DEVERR_INDEX);
    return a.n_keys;
}

__global__ void __launch_bounds__(kSortWarps * 32, 1) route_sort_kernel(const SortArgs a) {
    extern __shared__ int32_t smem[];
    int32_t(*hist)[kBins] = reinterpret_cast<int32_t(*)[kBins]>(smem);  // [warps][kBins]
    int32_t* total = smem + kSortWarps * kBins;                        // [kBins]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = ((a.n + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int f0 = min(a.n, warp * piece), f1 = min(a.n, f0 + piece);
    const uint32_t below = (1u << lane) - 1u;
    if (a.passes > 1)
        for (int e = threadIdx.x; e <= a.n_keys; e += blockDim.x) a.offsets[e] = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * kDigitBits;
        const bool last = pass + 1 == a.passes;
        const int32_t* src_key = a.key_buf[(pass + 1) & 1];
        const int32_t* src_idx = a.idx_buf[(pass + 1) & 1];
        for (int b = lane; b < kBins; b += 32) hist[warp][b] = 0;
        __syncwarp();
        for (int i = f0; i < f1; i += 32) {
            const bool live = i + lane < f1;
            int digit = -1;
            if (live) {
                const int32_t key = pass ? src_key[i + lane] : load_key(a, i + lane);
                digit = (key >> shift) & (kBins - 1);
            }
            const uint32_t peers = __match_any_sync(0xffffffffu, digit);
            if (live && (peers & below) == 0) hist[warp][digit] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        for (int b = threadIdx.x; b < kBins; b += blockDim.x) {
            int32_t s = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const int32_t c = hist[w][b];
                hist[w][b] = s;
                s += c;
            }
            total[b] = s;
        }
        __syncthreads();
        if (warp == 0) {  // exclusive sums over the digits, 16 per lane
            int32_t s = 0;
            for (int i = 0; i < kBins / 32; ++i) s += total[lane * (kBins / 32) + i];
            int32_t run = s;
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xffffffffu, run, d);
                if (lane >= d) run += o;
            }
            run -= s;
            for (int i = 0; i < kBins / 32; ++i) {
                const int32_t c = total[lane * (kBins / 32) + i];
                total[lane * (kBins / 32) + i] = run;
                run += c;
            }
        }
        __syncthreads();
        if (a.passes == 1)
            for (int b = threadIdx.x; b <= a.n_keys; b += blockDim.x) a.offsets[b] = total[b];
        for (int i = f0; i < f1; i += 32) {
            const bool live = i + lane < f1;
            int digit = -1;
            int32_t key = 0, f = 0;
            if (live) {
                key = pass ? src_key[i + lane] : load_key(a, i + lane);
                f = pass ? src_idx[i + lane] : i + lane;
                digit = (key >> shift) & (kBins - 1);
                if (a.passes > 1 && pass == 0) atomicAdd(a.offsets + key, 1);
            }
            const uint32_t peers = __match_any_sync(0xffffffffu, digit);
            int32_t p = 0;
            if (live) p = total[digit] + hist[warp][digit] + __popc(peers & below);
            __syncwarp();
            if (live && (peers & below) == 0) hist[warp][digit] += __popc(peers);
            __syncwarp();
            if (!live) continue;
            if (last) {
                a.order[p] = f;
                a.pos[f] = key < a.n_keys ? p : -1;
            } else {
                a.key_buf[pass & 1][p] = key;
                a.idx_buf[pass & 1][p] = f;
            }
        }
        __syncthreads();
    }
    if (a.passes > 1) {  // offsets holds the counts: exclusive sums in place, a block of threads at a time
        int32_t carry = 0;
        for (int e0 = 0; e0 <= a.n_keys; e0 += blockDim.x) {
            const int e = e0 + threadIdx.x;
            const int32_t c = e <= a.n_keys ? __ldcg(a.offsets + e) : 0;
            int32_t run = c;
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xffffffffu, run, d);
                if (lane >= d) run += o;
            }
            if (lane == 31) total[warp] = run;
            __syncthreads();
            int32_t before = carry, all = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                if (w < warp) before += total[w];
                all += total[w];
            }
            if (e <= a.n_keys) a.offsets[e] = before + run - c;
            carry += all;
            __syncthreads();
        }
    }
}

constexpr int kSortSmem = (kSortWarps + 1) * kBins * 4;

// ---------------------------------------------------------------- rows
struct RowArgs {
    const int32_t *order, *pos, *offsets;
    int64_t T, H, n_keys;
    int32_t k;
    const void *a, *b;  // operands (dispatch: x; combine: ys; gradient: dy, ys)
    int64_t lda, ldb;
    const float* w;     // [T][k] or null
    void* out;
    int64_t ldo;
    float* dw;          // [T][k]
};

// Rows past the last kept place are written as zeros, spread over the grid.
template <typename T, int V>
__device__ __forceinline__ void zero_tail(const RowArgs& a, T* out) {
    for (int64_t p = a.offsets[a.n_keys] + blockIdx.x; p < a.T * a.k; p += gridDim.x)
        for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V)
            Vec<T, V>::store(out + p * a.ldo + c, Vec<T, V>::zero());
}

// One CTA per token: its row is read once and written at its k places.
template <typename T, int V>
__global__ void dispatch_kernel(const RowArgs a) {
    using X = Vec<T, V>;
    const T* x = static_cast<const T*>(a.a) + blockIdx.x * a.lda;
    T* out = static_cast<T*>(a.out);
    const int32_t* pos = a.pos + static_cast<int64_t>(blockIdx.x) * a.k;
    for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) {
        const typename X::Raw v = X::load(x + c);
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = pos[j];
            if (p >= 0) X::store(out + p * a.ldo + c, v);
        }
    }
    zero_tail<T, V>(a, out);
}

// One CTA per token: its k rows summed in fp32 with their weights, rounded once.
template <typename T, int V>
__global__ void combine_kernel(const RowArgs a) {
    using X = Vec<T, V>;
    const T* ys = static_cast<const T*>(a.a);
    T* y = static_cast<T*>(a.out) + blockIdx.x * a.ldo;
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * a.k;
    for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) {
        float acc[V] = {};
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = a.pos[f0 + j];
            if (p < 0) continue;
            const float w = a.w ? a.w[f0 + j] : 1.f;
            float v[V];
            X::unpack(X::load(ys + p * a.lda + c), v);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(w, v[i], acc[i]);
        }
        X::store(y + c, X::pack(acc));
    }
}

// One CTA per token: for each of its k places dys = w dy and the dot product of
// dy with ys, summed in fp32 over the CTA.
template <typename T, int V>
__global__ void combine_grad_kernel(const RowArgs a) {
    using X = Vec<T, V>;
    __shared__ float part[32];
    const T* dy = static_cast<const T*>(a.a) + blockIdx.x * a.lda;
    const T* ys = static_cast<const T*>(a.b);
    T* dys = static_cast<T*>(a.out);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * a.k;
    for (int j = 0; j < a.k; ++j) {
        const int64_t p = a.pos[f0 + j];
        const float w = a.w ? a.w[f0 + j] : 1.f;
        float dot = 0.f;
        if (p >= 0) {
            for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V) {
                float d[V], v[V];
                X::unpack(X::load(dy + c), d);
                X::unpack(X::load(ys + p * a.ldb + c), v);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dot = fmaf(d[i], v[i], dot);
                    d[i] *= w;
                }
                X::store(dys + p * a.ldo + c, X::pack(d));
            }
        }
        for (int s = 16; s; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0 && a.dw) {
            float s = 0.f;
            for (int i = 0; i < (blockDim.x + 31) / 32; ++i) s += part[i];
            a.dw[f0 + j] = s;
        }
        __syncthreads();
    }
    zero_tail<T, V>(a, dys);
}

int row_threads(int64_t H, int v) {
    const int64_t n = (H + v - 1) / v;
    return n >= 512 ? 512 : static_cast<int>((n + 31) / 32 * 32);
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int32_t k, int64_t n_keys) {
    return n_keys < kBins ? 0 : static_cast<size_t>(T) * k * 16;
}

spmm_status launch_build_route(const void* ids, int32_t id_bytes, int64_t ldi, const spmm_route_t* R, void* ws,
                               cudaStream_t s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return SPMM_ERR_CUDA;
    if (!set_smem_attr_once(reinterpret_cast<const void*>(route_sort_kernel), kSortSmem, kSlotRouteSort))
        return SPMM_ERR_CUDA;
    const int32_t n = static_cast<int32_t>(R->T * R->k);
    SortArgs a{};
    a.ids = ids;
    a.ldi = ldi;
    a.wide = id_bytes == 8;
    a.k = R->k;
    a.n = n;
    a.n_keys = static_cast<int32_t>(R->n_keys);
    a.passes = 1;
    while (a.passes * kDigitBits < 31 && (R->n_keys >> (a.passes * kDigitBits))) ++a.passes;
    a.order = R->order;
    a.pos = R->pos;
    a.offsets = R->offsets;
    int32_t* w = static_cast<int32_t*>(ws);
    for (int i = 0; i < 2 && w; ++i) {
        a.key_buf[i] = w + static_cast<int64_t>(2 * i) * n;
        a.idx_buf[i] = w + static_cast<int64_t>(2 * i + 1) * n;
    }
    a.err = dev->err;
    trace_begin(SPMM_KERNEL_ROUTE, s);
    route_sort_kernel<<<1, kSortWarps * 32, kSortSmem, s>>>(a);
    trace_end(SPMM_KERNEL_ROUTE, s);
    return cuda_status(cudaGetLastError());
}

static RowArgs row_args(const spmm_route_t* R, int64_t H) {
    RowArgs a{};
    a.order = R->order;
    a.pos = R->pos;
    a.offsets = R->offsets;
    a.T = R->T;
    a.k = R->k;
    a.n_keys = R->n_keys;
    a.H = H;
    return a;
}

spmm_status launch_dispatch(const spmm_route_t* R, const void* x, int64_t ldx, void* xs, int64_t ldxs, int64_t H,
                            int32_t dtype, cudaStream_t s) {
    RowArgs a = row_args(R, H);
    a.a = x;
    a.lda = ldx;
    a.out = xs;
    a.ldo = ldxs;
    const int es = row_elem_bytes(dtype);
    const bool v = rows16(x, ldx, H, es) && rows16(xs, ldxs, H, es);
    const unsigned grid = static_cast<unsigned>(R->T);
    const int threads = row_threads(H, v ? 16 / es : 1);
    trace_begin(SPMM_KERNEL_ROWS, s);
    SPMM_ROWS_TYPED(dtype, v, dispatch_kernel, grid, threads, s, a);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(cudaGetLastError());
}

spmm_status launch_combine(const spmm_route_t* R, const void* ys, int64_t ldys, const float* w, void* y, int64_t ldy,
                           int64_t H, int32_t dtype, cudaStream_t s) {
    RowArgs a = row_args(R, H);
    a.a = ys;
    a.lda = ldys;
    a.w = w;
    a.out = y;
    a.ldo = ldy;
    const int es = row_elem_bytes(dtype);
    const bool v = rows16(ys, ldys, H, es) && rows16(y, ldy, H, es);
    const unsigned grid = static_cast<unsigned>(R->T);
    const int threads = row_threads(H, v ? 16 / es : 1);
    trace_begin(SPMM_KERNEL_ROWS, s);
    SPMM_ROWS_TYPED(dtype, v, combine_kernel, grid, threads, s, a);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(cudaGetLastError());
}

spmm_status launch_combine_grad(const spmm_route_t* R, const void* dy, int64_t lddy, const void* ys, int64_t ldys,
                                const float* w, void* dys, int64_t lddys, float* dw, int64_t H, int32_t dtype,
                                cudaStream_t s) {
    RowArgs a = row_args(R, H);
    a.a = dy;
    a.lda = lddy;
    a.b = ys;
    a.ldb = ldys;
    a.w = w;
    a.out = dys;
    a.ldo = lddys;
    a.dw = dw;
    const int es = row_elem_bytes(dtype);
    const bool v = rows16(dy, lddy, H, es) && rows16(ys, ldys, H, es) && rows16(dys, lddys, H, es);
    const unsigned grid = static_cast<unsigned>(R->T);
    const int threads = row_threads(H, v ? 16 / es : 1);
    trace_begin(SPMM_KERNEL_ROWS, s);
    SPMM_ROWS_TYPED(dtype, v, combine_grad_kernel, grid, threads, s, a);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(cudaGetLastError());
}

}  // namespace spmm
