// experts.cu -- the experts' products on rows sorted by expert: one block-
// diagonal sparse x dense product and its two gradients.  Rows offsets[e] ..
// offsets[e + 1] - 1 belong to expert e with weights W[e] (N x K):
//   forward   ys[p]  = W[e] xs[p]
//   dx        dxs[p] = W[e]^T dys[p]
//   dw        dW[e]  = sum_p dys[p] xs[p]^T
// Sums are fp32, rounded once to the operands' type.
#include "internal.h"
#include "rowvec.cuh"

namespace spmm {
namespace {

using namespace rows;

constexpr int kTile = 64, kDepth = 16;

// One operand element (r, d): address base + r * rs + d * ds.
struct Operand {
    const void* p;
    int64_t rs, ds;
};

template <typename T>
__device__ void product_tile(const Operand A, const Operand B, int64_t m0, int64_t M, int64_t n0, int64_t N, int64_t D,
                             T* C, int64_t ldc, float (*sa)[kTile + 1], float (*sb)[kTile + 1]) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int64_t d0 = 0; d0 < D; d0 += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
            // the contiguous direction of each operand varies fastest
            const int ra = A.ds == 1 ? i / kDepth : i % kTile, da = A.ds == 1 ? i % kDepth : i / kTile;
            const int rb = B.ds == 1 ? i / kDepth : i % kTile, db = B.ds == 1 ? i % kDepth : i / kTile;
            sa[da][ra] = m0 + ra < M && d0 + da < D
                             ? to_f32(static_cast<const T*>(A.p)[(m0 + ra) * A.rs + (d0 + da) * A.ds]) : 0.f;
            sb[db][rb] = n0 + rb < N && d0 + db < D
                             ? to_f32(static_cast<const T*>(B.p)[(n0 + rb) * B.rs + (d0 + db) * B.ds]) : 0.f;
        }
        __syncthreads();
        for (int d = 0; d < kDepth; ++d)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[d][ty + 16 * i], sb[d][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (m0 + ty + 16 * i < M && n0 + tx + 16 * j < N)
                C[(m0 + ty + 16 * i) * ldc + n0 + tx + 16 * j] = from_f32<T>(acc[i][j]);
}

struct ExpertArgs {
    const int32_t* offsets;
    int64_t E, R, rows_d, cols;  // depth of a row product, columns of the result
    const void *rows, *w;
    int64_t ldr, ldw, w_rs, w_ds, w_es;
    void* out;
    int64_t ldo;
};

// Row products (forward, dx): grid (column tiles, experts).
template <typename T>
__global__ void __launch_bounds__(256) rows_kernel(const ExpertArgs a) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    const int64_t e = blockIdx.y, p0 = a.offsets[e], p1 = a.offsets[e + 1];
    const Operand A{static_cast<const T*>(a.rows) + p0 * a.ldr, a.ldr, 1};
    const Operand B{static_cast<const T*>(a.w) + e * a.w_es, a.w_rs, a.w_ds};
    T* C = static_cast<T*>(a.out) + p0 * a.ldo;
    for (int64_t m0 = 0; m0 < p1 - p0; m0 += kTile)
        product_tile<T>(A, B, m0, p1 - p0, static_cast<int64_t>(blockIdx.x) * kTile, a.cols, a.rows_d, C, a.ldo, sa, sb);
    // rows of dropped choices are written as zeros, by the first expert's CTAs
    if (e == 0)
        for (int64_t p = a.offsets[a.E]; p < a.R; ++p)
            for (int64_t c = static_cast<int64_t>(blockIdx.x) * kTile + threadIdx.x;
                 c < a.cols && c < (static_cast<int64_t>(blockIdx.x) + 1) * kTile; c += blockDim.x)
                static_cast<T*>(a.out)[p * a.ldo + c] = from_f32<T>(0.f);
}

struct DwArgs {
    const int32_t* offsets;
    int64_t N, K;
    const void *dys, *xs;
    int64_t ldd, ldx;
    void* dW;
    int64_t ldw, w_es;
};

// Weight gradients: grid (K tiles, N tiles, experts).
template <typename T>
__global__ void __launch_bounds__(256) dw_kernel(const DwArgs a) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    const int64_t e = blockIdx.z, p0 = a.offsets[e], p1 = a.offsets[e + 1];
    const Operand A{static_cast<const T*>(a.dys) + p0 * a.ldd, 1, a.ldd};
    const Operand B{static_cast<const T*>(a.xs) + p0 * a.ldx, 1, a.ldx};
    product_tile<T>(A, B, static_cast<int64_t>(blockIdx.y) * kTile, a.N, static_cast<int64_t>(blockIdx.x) * kTile, a.K,
                    p1 - p0, static_cast<T*>(a.dW) + e * a.w_es, a.ldw, sa, sb);
}

unsigned tiles(int64_t n) { return static_cast<unsigned>((n + kTile - 1) / kTile); }

}  // namespace

spmm_status launch_experts_rows(const spmm_route_t* R, const void* rows, int64_t ldr, const void* W, int64_t ldw,
                                int64_t lde, int64_t N, int64_t K, bool transposed, int32_t dtype, void* out, int64_t ldo,
                                cudaStream_t s) {
    ExpertArgs a{};
    a.offsets = R->offsets;
    a.E = R->n_keys;
    a.R = R->T * R->k;
    a.rows_d = transposed ? N : K;
    a.cols = transposed ? K : N;
    a.rows = rows;
    a.ldr = ldr;
    a.w = W;
    a.w_rs = transposed ? 1 : ldw;
    a.w_ds = transposed ? ldw : 1;
    a.w_es = lde;
    a.out = out;
    a.ldo = ldo;
    const dim3 grid(tiles(a.cols), static_cast<unsigned>(a.E));
    trace_begin(SPMM_KERNEL_EXPERTS, s);
    if (dtype == SPMM_BF16)
        rows_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
    else
        rows_kernel<__half><<<grid, 256, 0, s>>>(a);
    trace_end(SPMM_KERNEL_EXPERTS, s);
    return cuda_status(cudaGetLastError());
}

spmm_status launch_experts_dw(const spmm_route_t* R, const void* dys, int64_t ldd, const void* xs, int64_t ldx,
                              int64_t N, int64_t K, int32_t dtype, void* dW, int64_t ldw, int64_t lde, cudaStream_t s) {
    DwArgs a{R->offsets, N, K, dys, xs, ldd, ldx, dW, ldw, lde};
    const dim3 grid(tiles(K), tiles(N), static_cast<unsigned>(R->n_keys));
    trace_begin(SPMM_KERNEL_EXPERTS, s);
    if (dtype == SPMM_BF16)
        dw_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
    else
        dw_kernel<__half><<<grid, 256, 0, s>>>(a);
    trace_end(SPMM_KERNEL_EXPERTS, s);
    return cuda_status(cudaGetLastError());
}

}  // namespace spmm
