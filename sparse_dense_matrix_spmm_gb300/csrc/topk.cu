// topk.cu -- the router of a mixture of experts: each token's k largest logits with
// their softmax weights, and the gradient of the weights for the logits.
// A warp per token: its E logits stay in registers as order-preserving integers, and
// k times the warp takes the largest (two warp-wide integer reductions: the value,
// then the lowest index that has it).  The logits are read once, and what a router
// costs is the latency of these rounds and of the launch: E = 128 bf16 for 16384 tokens
// are 4 MB.
#include "internal.h"
#include "rowvec.cuh"

namespace spmm {
namespace {

using namespace rows;

constexpr int kWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;
constexpr uint32_t kLowest = 0x007FFFFFu;  // -infinity as an ordered integer: never chosen

struct TopkArgs {
    const void* logits;
    int64_t ldl;
    int64_t T;
    int32_t E, k;
    int32_t renorm;
    void* ids;
    int32_t wide;
    float* w;
    const float* dw;
    void* dlogits;
    int64_t ldd;
    int* err;
};

// Integers in the order of the values: -0 equals +0, every NaN is above +infinity.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = +0
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);  // all ones: a NaN
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// Lane l holds logits l, l + 32, ..: N of them, 0 in place of what cannot be chosen.
template <typename T, int N>
__device__ __forceinline__ uint32_t load_keys(const T* row, int E, int lane, uint32_t (&key)[N]) {
    T raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane + 32 * i < E) raw[i] = row[lane + 32 * i];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        key[i] = lane + 32 * i < E ? ordered(to_f32<T>(raw[i])) : 0u;
        if (key[i] <= kLowest) key[i] = 0u;
        most = max(most, key[i]);
    }
    return __reduce_max_sync(kAll, most);
}
// The sum of exp(logit - top) over all logits.
template <int N>
__device__ __forceinline__ float exp_sum(const uint32_t (&key)[N], float top) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (key[i]) z += expf(value_of(key[i]) - top);
    return warp_sum(z);
}

template <typename T, int N>
__global__ void __launch_bounds__(kWarps * 32) topk_kernel(const TopkArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    uint32_t key[N];
    const uint32_t first = load_keys<T, N>(static_cast<const T*>(a.logits) + t * a.ldl, a.E, lane, key);
    const float top = value_of(first);
    float z = 0.f;
    if (!a.renorm && first) z = exp_sum<N>(key, top);
    uint32_t mine = 0;  // lane j keeps choice j
    int id = -1;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t m = __reduce_max_sync(kAll, best);
        if (m == 0) break;
        const uint32_t index = static_cast<uint32_t>(lane + 32 * at);
        const uint32_t chosen = __reduce_min_sync(kAll, best == m ? index : 0xFFFFFFFFu);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (chosen == static_cast<uint32_t>(lane + 32 * i)) key[i] = 0u;
        if (lane == j) {
            mine = m;
            id = static_cast<int>(chosen);
        }
    }
    const float p = id >= 0 ? expf(value_of(mine) - top) : 0.f;
    if (a.renorm) z = warp_sum(p);
    if (lane < a.k) {
        const int64_t o = t * a.k + lane;
        if (a.wide)
            static_cast<int64_t*>(a.ids)[o] = id;
        else
            static_cast<int32_t*>(a.ids)[o] = id;
        a.w[o] = id >= 0 ? p / z : 0.f;
    }
}

// A warp per token writes -p_e sum_i w_i dw_i everywhere (zeros with renorm), then
// the chosen places again; __syncwarp orders the two.
template <typename T, int N>
__global__ void __launch_bounds__(kWarps * 32) topk_grad_kernel(const TopkArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    int64_t id = -1;
    if (lane < a.k) {
        const int64_t o = t * a.k + lane;
        id = a.wide ? static_cast<const int64_t*>(a.ids)[o] : static_cast<const int32_t*>(a.ids)[o];
        if (id >= a.E) {
            atomicOr(a.err, SPMM_DEVERR_INDEX);
            id = -1;
        }
    }
    const bool live = id >= 0;
    const float w = live ? a.w[t * a.k + lane] : 0.f;
    const float wd = live ? w * a.dw[t * a.k + lane] : 0.f;
    const float dot = warp_sum(wd);
    T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
    if (a.renorm) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < a.E) out[lane + 32 * i] = from_f32<T>(0.f);
    } else {
        uint32_t key[N];
        const uint32_t first = load_keys<T, N>(static_cast<const T*>(a.logits) + t * a.ldl, a.E, lane, key);
        const float top = value_of(first), z = exp_sum<N>(key, top);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < a.E)
                out[lane + 32 * i] = from_f32<T>(key[i] ? -(expf(value_of(key[i]) - top) / z) * dot : 0.f);
    }
    __syncwarp();
    // the chosen places; the same id more than once is added up by its first lane
    const uint32_t same = __match_any_sync(kAll, live ? id : -1 - static_cast<int64_t>(lane));
    float sum = wd, p = w;
    if (__any_sync(kAll, same & (same - 1))) {
        sum = p = 0.f;
        for (int l = 0; l < 32; ++l) {
            const float sl = __shfl_sync(kAll, wd, l), pl = __shfl_sync(kAll, w, l);
            if (same >> l & 1u) {
                sum += sl;
                p = a.renorm ? p + pl : pl;
            }
        }
    }
    if (live && __ffs(same) - 1 == lane) out[id] = from_f32<T>(sum - p * dot);
}

template <typename T>
cudaError_t launch_typed(const TopkArgs& a, bool grad, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((a.T + kWarps - 1) / kWarps));
    const int n = (a.E + 31) / 32;
#define SPMM_TOPK(N) \
    return launch_rows(grad ? topk_grad_kernel<T, N> : topk_kernel<T, N>, grid, kWarps * 32, s, a)
    if (n <= 1) SPMM_TOPK(1);
    if (n <= 2) SPMM_TOPK(2);
    if (n <= 4) SPMM_TOPK(4);
    if (n <= 8) SPMM_TOPK(8);
    if (n <= 16) SPMM_TOPK(16);
    SPMM_TOPK(32);
#undef SPMM_TOPK
}

spmm_status launch(const TopkArgs& a, int32_t dtype, bool grad, cudaStream_t s) {
    trace_begin(SPMM_KERNEL_TOPK, s);
    const cudaError_t e = dtype == SPMM_F32   ? launch_typed<float>(a, grad, s)
                          : dtype == SPMM_F16 ? launch_typed<__half>(a, grad, s)
                                              : launch_typed<__nv_bfloat16>(a, grad, s);
    trace_end(SPMM_KERNEL_TOPK, s);
    return cuda_status(e);
}

}  // namespace

spmm_status launch_topk(const void* logits, int64_t T, int64_t E, int64_t ldl, int32_t dtype, int32_t k, int32_t renorm,
                        void* ids, int32_t id_bytes, float* w, cudaStream_t s) {
    TopkArgs a{};
    a.logits = logits;
    a.ldl = ldl;
    a.T = T;
    a.E = static_cast<int32_t>(E);
    a.k = k;
    a.renorm = renorm;
    a.ids = ids;
    a.wide = id_bytes == 8;
    a.w = w;
    return launch(a, dtype, false, s);
}

spmm_status launch_topk_grad(const void* logits, int64_t T, int64_t E, int64_t ldl, int32_t dtype, int32_t k,
                             int32_t renorm, const void* ids, int32_t id_bytes, const float* w, const float* dw,
                             void* dlogits, int64_t ldd, cudaStream_t s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return SPMM_ERR_CUDA;
    TopkArgs a{};
    a.logits = logits;
    a.ldl = ldl;
    a.T = T;
    a.E = static_cast<int32_t>(E);
    a.k = k;
    a.renorm = renorm;
    a.ids = const_cast<void*>(ids);
    a.wide = id_bytes == 8;
    a.w = const_cast<float*>(w);
    a.dw = dw;
    a.dlogits = dlogits;
    a.ldd = ldd;
    a.err = dev->err;
    return launch(a, dtype, true, s);
}

}  // namespace spmm
