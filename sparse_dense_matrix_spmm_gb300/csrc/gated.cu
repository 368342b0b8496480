// gated.cu -- the experts' gated block on CUDA cores (up to 16 rows in all, or 64
// spread over as many experts), and the gradient of its activation.
//   forward   [g u] = W[e] xs[p],  h[p] = act(g) u
//   gradient  dgu[p] = [dh u act'(g), dh act(g)]
#include "gated.cuh"
#include "internal.h"
#include "rowvec.cuh"

namespace spmm {
namespace {

using namespace rows;
using namespace gated;

// ---------------------------------------------------------------- forward, very few rows
// Dot products on CUDA cores: a warp takes one feature, its gate row and its up
// row, with up to four rows of an expert, and has both sums in every lane at the
// end.  Where [g u] is kept in 8 bits a CTA's 16 warps are a group of 16 features
// and meet in shared memory; else 8 warps that do not wait for one another.  One
// token with 2 of 8 experts (2 x 2048 x 4096, 67 MB) 13.0 us, with 8 of 64 (2 x 768 x
// 2048, 50 MB) 10.7 us, with 8 of 128 (2 x 1280 x 4096, 168 MB) 28 us: launch, ramp
// and the chain of offsets, weights and shuffles, then HBM.
constexpr int kVecRows = 4;

struct VecArgs {
    const int32_t* offsets;
    int32_t E;
    const void *xs, *W;
    int64_t ldx, ldw, lde;
    int32_t N, K;
    GatedOut out;
};

// sums[half][row] of the gate row wg and the up row wu with C rows of x.
template <typename T, int C>
__device__ __forceinline__ void dot_rows(const VecArgs& a, const T* wg, const T* wu, const T* x, int lane,
                                         float (&sums)[2][kVecRows]) {
    using V = Vec<T, 8>;
    float acc[2][C] = {};
    // Loads per weight row before their sums: four keep a lone row's weights coming
    // (two: 13.0 -> 14.1, 28 -> 30.5 us), with more rows their registers are sums.
    constexpr int kFlight = C == 1 ? 4 : 2;
    for (int k0 = lane * 8; k0 < a.K; k0 += 256 * kFlight) {
        uint4 r[2][kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int k = k0 + 256 * i;
            r[0][i] = k < a.K ? ptx::ld_global_cs(reinterpret_cast<const uint4*>(wg + k)) : V::zero();
            r[1][i] = k < a.K ? ptx::ld_global_cs(reinterpret_cast<const uint4*>(wu + k)) : V::zero();
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int k = k0 + 256 * i;
            if (k >= a.K) break;
            float f0[8], f1[8];
            V::unpack(r[0][i], f0);
            V::unpack(r[1][i], f1);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float v[8];
                V::unpack(V::load(x + c * a.ldx + k), v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[0][c] = fmaf(f0[j], v[j], acc[0][c]);
                    acc[1][c] = fmaf(f1[j], v[j], acc[1][c]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int s = 16; s; s >>= 1) {
            acc[0][c] += __shfl_xor_sync(0xffffffffu, acc[0][c], s);
            acc[1][c] += __shfl_xor_sync(0xffffffffu, acc[1][c], s);
        }
        sums[0][c] = acc[0][c];
        sums[1][c] = acc[1][c];
    }
}

// Grid (features, sorted place): the CTAs of an expert's first place and of every
// fourth after it take up to four of its rows, the others leave; places of dropped
// choices are zeroed.
template <bool PACKED>
constexpr int kVecWarps = PACKED ? 16 : 8;
template <typename T, int ACT, bool PACKED>
__global__ void __launch_bounds__(kVecWarps<PACKED> * 32, 32 / kVecWarps<PACKED>)
    gated_vec_kernel(const VecArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = blockIdx.y, n = blockIdx.x * kVecWarps<PACKED> + warp;
    int rows = 1;
    float sums[2][kVecRows] = {};
    const bool live = p < a.offsets[a.E];
    if (live) {
        int lo = 0, hi = a.E;  // the last e with offsets[e] <= p, 32 probes at a time
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + step * lane;
            const uint32_t le = __ballot_sync(0xffffffffu, at < hi && a.offsets[at] <= p);
            lo += step * (31 - __clz(le));
            hi = min(hi, lo + step);
        }
        if ((p - a.offsets[lo]) % kVecRows) return;
        rows = min(kVecRows, a.offsets[lo + 1] - p);
        const T* x = static_cast<const T*>(a.xs) + p * a.ldx;
        const T* wg = static_cast<const T*>(a.W) + lo * a.lde + n * a.ldw;
        const T* wu = wg + a.N * a.ldw;
        if (rows == 1)
            dot_rows<T, 1>(a, wg, wu, x, lane, sums);
        else if (rows == 2)
            dot_rows<T, 2>(a, wg, wu, x, lane, sums);
        else if (rows == 3)
            dot_rows<T, 3>(a, wg, wu, x, lane, sums);
        else
            dot_rows<T, 4>(a, wg, wu, x, lane, sums);
    }
    // lane c writes row c
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int c = 0; c < kVecRows; ++c) {
        g = lane == c ? sums[0][c] : g;
        u = lane == c ? sums[1][c] : u;
    }
    if (lane < rows) {
        const int64_t row = p + lane;
        static_cast<T*>(a.out.h)[row * a.out.ldh + n] = from_f32<T>(live ? act<ACT>(g) * u : 0.f);
        if (!PACKED && a.out.gu) {
            T* gu = static_cast<T*>(a.out.gu) + row * a.out.ldgu + n;
            gu[0] = from_f32<T>(g);
            gu[a.N] = from_f32<T>(u);
        }
    }
    if constexpr (PACKED) {
        __shared__ float all[2][kVecRows][16];  // gate and up
        if (lane < kVecRows) {
            all[0][lane][warp] = g;
            all[1][lane][warp] = u;
        }
        __syncthreads();
        if (threadIdx.x >= 2 * kVecRows * 16) return;  // whole warps: half, row, feature
        const int f = threadIdx.x & 15, c = threadIdx.x >> 4 & 3, half = threadIdx.x >> 6;
        const float v = all[half][c][f];
        uint32_t code = magnitude_code(v);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) code = max(code, __shfl_xor_sync(0xffffffffu, code, d));
        const uint32_t b = scale_byte(code);
        const int64_t row = p + c, col = static_cast<int64_t>(half) * a.N + blockIdx.x * 16 + f;
        if (c < rows) {
            uint32_t q[1];
            quantise({v}, b, q);
            a.out.q[row * a.out.ldq + col] = static_cast<int8_t>(q[0]);
            if (f == 0) a.out.scale[row * a.out.lds + col / kGroup] = static_cast<uint8_t>(b);
        }
    }
}

// ---------------------------------------------------------------- gradient of the activation
// A thread takes 8 features of a place, reads dh, g and u and writes both gradients (and
// h).  Bound by HBM from rows (16372 x 1280 bf16, 210 MB: 31 us; 16382 x 1792, 294 MB: 43
// us) and, but for gelu, from 8 bits (silu 170 MB: 26 us, 238 MB: 35 us; tanh form 28 and
// 38 us, gelu 30 and 41 us, by instructions).  A thread's row by one multiplication:
// with divisions 26.6, 36, 28.2, 38.4, 31.3 and 43 us from 8 bits.
constexpr int kGradThreads = 256;

struct GradArgs {
    const int32_t* offsets;
    int32_t E;
    int64_t R;
    int32_t N;
    uint64_t per_row;  // 2^64 over the threads of a row, rounded up
    const void* dh;
    int64_t lddh;
    const void* gu;
    int64_t ldgu;
    const int8_t* q;
    int64_t ldq;
    const uint8_t* scale;
    int64_t lds;
    void* dgu;
    int64_t lddgu;
    void* h;
    int64_t ldh;
};

// Eight kept values in 8 bits (half a group).
__device__ __forceinline__ void unpack8(const uint2& q, uint32_t byte, float (&f)[8]) {
    const float unit = unit_of(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = byte_of((i < 4 ? q.x : q.y) ^ 0x80808080u, i & 3) * unit;
}

// Threads take 8 features each in the order of rows and features, so that none idles
// whatever N is.  Loads come before the test for rows past the kept ones (they lie
// inside the operands; what they hold is not used).
template <typename T, int ACT, bool PACKED, bool H>
__global__ void __launch_bounds__(kGradThreads) gated_grad_kernel(const GradArgs a) {
    using V = Vec<T, 8>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    // exact while threads x threads of a row stay below 2^64 (the launcher refuses more)
    const uint64_t thread = static_cast<uint64_t>(blockIdx.x) * kGradThreads + threadIdx.x;
    const int64_t p = static_cast<int64_t>(__umul64hi(thread, a.per_row));
    // modulo 2^32, which the place in a row lies below: rows x features may be more
    const uint32_t before = static_cast<uint32_t>(p) * static_cast<uint32_t>(a.N / 8);
    const int c = static_cast<int>(static_cast<uint32_t>(thread) - before) * 8;
    if (p >= a.R) return;
    const typename V::Raw rd = V::load(static_cast<const T*>(a.dh) + p * a.lddh + c);
    typename V::Raw rg, ru;
    uint2 qg, qu;
    uint32_t sg = 1, su = 1;
    if (PACKED) {
        const int8_t* q = a.q + p * a.ldq + c;
        const uint8_t* s = a.scale + p * a.lds + c / kGroup;
        qg = *reinterpret_cast<const uint2*>(q);
        qu = *reinterpret_cast<const uint2*>(q + a.N);
        sg = s[0];
        su = s[a.N / kGroup];
    } else {
        const T* r = static_cast<const T*>(a.gu) + p * a.ldgu + c;
        rg = V::load(r);
        ru = V::load(r + a.N);
    }
    float d[8] = {}, f[8] = {}, y[8] = {};
    if (p < a.offsets[a.E]) {
        float g[8], u[8];
        V::unpack(rd, d);
        if (PACKED) {
            unpack8(qg, sg, g);
            unpack8(qu, su, u);
        } else {
            V::unpack(rg, g);
            V::unpack(ru, u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v, dv;
            act_grad<ACT>(g[i], v, dv);
            f[i] = d[i] * v;
            d[i] *= u[i] * dv;
            if (H) y[i] = v * u[i];
        }
    }
    T* dg = static_cast<T*>(a.dgu) + p * a.lddgu + c;
    V::store(dg, V::pack(d));
    V::store(dg + a.N, V::pack(f));
    if (H) V::store(static_cast<T*>(a.h) + p * a.ldh + c, V::pack(y));
}

template <typename T, int ACT, bool PACKED>
cudaError_t launch_grad_of(const GradArgs& a, int64_t blocks, cudaStream_t s) {
    return launch_rows(a.h ? gated_grad_kernel<T, ACT, PACKED, true> : gated_grad_kernel<T, ACT, PACKED, false>,
                       dim3(static_cast<unsigned>(blocks)), kGradThreads, s, a);
}
template <typename T, bool PACKED>
cudaError_t launch_grad(const GradArgs& a, int64_t blocks, int32_t act, cudaStream_t s) {
    if (act == SPMM_ACT_SILU) return launch_grad_of<T, SPMM_ACT_SILU, PACKED>(a, blocks, s);
    if (act == SPMM_ACT_GELU) return launch_grad_of<T, SPMM_ACT_GELU, PACKED>(a, blocks, s);
    return launch_grad_of<T, SPMM_ACT_GELU_TANH, PACKED>(a, blocks, s);
}

template <typename T, bool PACKED>
cudaError_t launch_vec_of(const VecArgs& a, int64_t rows, int32_t act, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.N / kVecWarps<PACKED>), static_cast<unsigned>(rows));
    return launch_rows(act == SPMM_ACT_SILU   ? gated_vec_kernel<T, SPMM_ACT_SILU, PACKED>
                       : act == SPMM_ACT_GELU ? gated_vec_kernel<T, SPMM_ACT_GELU, PACKED>
                                              : gated_vec_kernel<T, SPMM_ACT_GELU_TANH, PACKED>,
                       grid, kVecWarps<PACKED> * 32, s, a);
}
template <typename T>
cudaError_t launch_vec(const VecArgs& a, int64_t rows, int32_t act, cudaStream_t s) {
    return a.out.q ? launch_vec_of<T, true>(a, rows, act, s) : launch_vec_of<T, false>(a, rows, act, s);
}

}  // namespace

spmm_status launch_experts_gated_vec(const spmm_route_t* R, const void* xs, int64_t ldx, const void* W, int64_t ldw,
                                     int64_t lde, int64_t N, int64_t K, int32_t dtype, int32_t act, const GatedOut& out,
                                     cudaStream_t s) {
    const VecArgs a{R->offsets, static_cast<int32_t>(R->n_keys), xs, W, ldx, ldw, lde, static_cast<int32_t>(N),
                    static_cast<int32_t>(K), out};
    const int64_t rows = R->T * R->k;
    trace_begin(SPMM_KERNEL_EXPERTS, s);
    const cudaError_t e = dtype == SPMM_BF16 ? launch_vec<__nv_bfloat16>(a, rows, act, s) : launch_vec<__half>(a, rows, act, s);
    trace_end(SPMM_KERNEL_EXPERTS, s);
    return cuda_status(e);
}

spmm_status launch_gated_grad(const spmm_route_t* R, const void* dh, int64_t lddh, const void* gu, int64_t ldgu,
                              const spmm_rows8_t* packed, int64_t N, int32_t dtype, int32_t act, void* dgu,
                              int64_t lddgu, void* h, int64_t ldh, cudaStream_t s) {
    GradArgs a{};
    a.offsets = R->offsets;
    a.E = static_cast<int32_t>(R->n_keys);
    a.R = R->T * R->k;
    a.N = static_cast<int32_t>(N);
    a.per_row = UINT64_MAX / static_cast<uint64_t>(N / 8) + 1;  // N % 16 == 0
    a.dh = dh;
    a.lddh = lddh;
    a.gu = gu;
    a.ldgu = ldgu;
    if (packed) {
        a.q = packed->q;
        a.ldq = packed->ldq;
        a.scale = packed->scale;
        a.lds = packed->lds;
    }
    a.dgu = dgu;
    a.lddgu = lddgu;
    a.h = h;
    a.ldh = ldh;
    const int64_t blocks = (a.R * (N / 8) + kGradThreads - 1) / kGradThreads;
    if (blocks >= int64_t(1) << 31 || static_cast<uint64_t>(blocks) * kGradThreads > UINT64_MAX / static_cast<uint64_t>(N / 8))
        return SPMM_ERR_UNSUPPORTED;  // 8 TB of dgu and more
    cudaError_t e;
    trace_begin(SPMM_KERNEL_GATED_GRAD, s);
    if (dtype == SPMM_BF16)
        e = packed ? launch_grad<__nv_bfloat16, true>(a, blocks, act, s) : launch_grad<__nv_bfloat16, false>(a, blocks, act, s);
    else
        e = packed ? launch_grad<__half, true>(a, blocks, act, s) : launch_grad<__half, false>(a, blocks, act, s);
    trace_end(SPMM_KERNEL_GATED_GRAD, s);
    return cuda_status(e);
}

}  // namespace spmm
