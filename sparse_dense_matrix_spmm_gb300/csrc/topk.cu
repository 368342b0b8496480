// topk.cu -- the router of a mixture of experts: each token's k largest logits with
// their softmax weights, and the gradient of the weights for the logits.
// A warp per token: its E logits stay in registers as order-preserving integers, and
// k times the warp takes the largest.  Done on all of them a round costs about 6
// instructions per 32 experts (256 experts, k = 8: 16.4 us for 16384 tokens).  So the
// logits are thinned first: the k-th largest of the 32 lanes' maxima is at most the k-th
// largest of all, so whatever lies below it cannot be chosen, and what is left, mostly
// little more than k, moves to one logit per lane.  A round is then two warp-wide
// integer reductions, the largest logit and the lowest index that has it.  With many
// equal logits more than 32 may be left; then the rounds run over all of them.
// The logits are read once; E = 256 fp32 for 16384 tokens are 16.8 MB, 2.5 us of HBM, and
// the kernel takes 9.4 us, bound by instructions.
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

// Integers in the order of the values.  The sum with zero makes +0 of -0 and the one
// positive NaN of every NaN, which so lies above +infinity.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);  // all ones: a NaN
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// Lane l holds logits l, l + 32, ..: N of them, -infinity past the last.  Returns the largest.
template <typename T, int N>
__device__ __forceinline__ uint32_t load_keys(const T* row, int E, int lane, uint32_t (&key)[N]) {
    T raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane + 32 * i < E) raw[i] = row[lane + 32 * i];
    uint32_t most = kLowest;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        key[i] = lane + 32 * i < E ? ordered(to_f32<T>(raw[i])) : kLowest;
        most = max(most, key[i]);
    }
    return most;
}
// The sum of exp(logit - top) over all logits, of which one at least is not -infinity.
template <int N>
__device__ __forceinline__ float exp_sum(const uint32_t (&key)[N], float top) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) z += expf(value_of(key[i]) - top);
    return warp_sum(z);
}

template <typename T, int N>
__global__ void __launch_bounds__(kWarps * 32) topk_kernel(const TopkArgs a) {
    __shared__ uint2 thinned[kWarps][32];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    uint2* kept = thinned[threadIdx.x >> 5];
    uint32_t key[N];
    uint32_t head = load_keys<T, N>(static_cast<const T*>(a.logits) + t * a.ldl, a.E, lane, key);
    const uint32_t first = __reduce_max_sync(kAll, head);
    const float top = value_of(first);
    float z = 0.f;
    if (!a.renorm && first > kLowest) z = exp_sum<N>(key, top);
    uint32_t mine = 0;  // lane j keeps choice j
    int id = -1;
    uint32_t one = key[0], index = lane;  // a logit per lane, and its index
    int left = 32;
    if constexpr (N > 1) {
        // the k-th largest of the lanes' maxima, above -infinity
        uint32_t least = first;
        for (int n = 0;;) {
            const uint32_t equal = __ballot_sync(kAll, head == least);
            n += __popc(equal);
            if (n >= a.k) break;
            if (head == least) head = 0u;
            least = __reduce_max_sync(kAll, head);
            if (least == 0u) break;
        }
        least = max(least, kLowest + 1u);
        int mine_left = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) mine_left += key[i] >= least;
        int place = mine_left;  // becomes the sum over the lanes up to this one
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(kAll, place, d);
            if (lane >= d) place += o;
        }
        left = __shfl_sync(kAll, place, 31);
        if (left <= 32) {
            place -= mine_left;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (key[i] >= least) kept[place++] = make_uint2(key[i], lane + 32 * i);
            __syncwarp();
            const uint2 v = lane < left ? kept[lane] : make_uint2(0u, 0u);
            one = v.x;
            index = v.y;
        }
    }
    if (left <= 32) {
        for (int j = 0; j < a.k; ++j) {
            const uint32_t m = __reduce_max_sync(kAll, one);
            if (m <= kLowest) break;
            const uint32_t chosen = __reduce_min_sync(kAll, one == m ? index : 0xFFFFFFFFu);
            if (index == chosen) one = 0u;
            if (lane == j) {
                mine = m;
                id = static_cast<int>(chosen);
            }
        }
    } else {
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
            if (m <= kLowest) break;
            const uint32_t chosen =
                __reduce_min_sync(kAll, best == m ? static_cast<uint32_t>(lane + 32 * at) : 0xFFFFFFFFu);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (chosen == static_cast<uint32_t>(lane + 32 * i)) key[i] = 0u;
            if (lane == j) {
                mine = m;
                id = static_cast<int>(chosen);
            }
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
// the chosen places again; __syncwarp orders the two.  (256 experts, k = 8, 16384 tokens:
// 4.7 us.)
template <typename T, int N>
__global__ void __launch_bounds__(kWarps * 32) topk_grad_kernel(const TopkArgs a) {
    __shared__ uint32_t owners[kWarps][32 * N];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    int64_t id = -1;
    float w = 0.f, wd = 0.f;
    if (lane < a.k) {
        const int64_t o = t * a.k + lane;
        w = a.w[o];
        wd = a.dw[o];
        id = a.wide ? static_cast<const int64_t*>(a.ids)[o] : static_cast<const int32_t*>(a.ids)[o];
        if (id >= a.E) {
            atomicOr(a.err, SPMM_DEVERR_INDEX);
            id = -1;
        }
    }
    const bool live = id >= 0;
    w = live ? w : 0.f;  // a dropped choice's may be anything
    wd = live ? w * wd : 0.f;
    const float dot = warp_sum(wd);
    T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
    if (a.renorm) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < a.E) out[lane + 32 * i] = from_f32<T>(0.f);
    } else {
        uint32_t key[N];
        const uint32_t first =
            __reduce_max_sync(kAll, load_keys<T, N>(static_cast<const T*>(a.logits) + t * a.ldl, a.E, lane, key));
        const float top = value_of(first), z = exp_sum<N>(key, top);
        // a token without experts: z is NaN, and every entry 0
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < a.E)
                out[lane + 32 * i] = from_f32<T>(first > kLowest ? -(expf(value_of(key[i]) - top) / z) * dot : 0.f);
    }
    __syncwarp();
    // The chosen places.  The same id more than once, which spmm_topk never gives: a lane
    // that does not find itself where it left its number tells (a warp-wide match of all
    // ids costs more than the rest of the kernel); its first lane then adds up.
    uint32_t* owner = owners[threadIdx.x >> 5];
    if (live) owner[id] = static_cast<uint32_t>(lane);
    __syncwarp();
    float sum = wd, p = w;
    bool first = live;
    if (__any_sync(kAll, live && owner[id] != static_cast<uint32_t>(lane))) {
        const uint32_t same = __match_any_sync(kAll, live ? static_cast<int>(id) : -1 - lane);
        first = live && __ffs(same) - 1 == lane;
        sum = p = 0.f;
        for (int l = 0; l < 32; ++l) {
            const float sl = __shfl_sync(kAll, wd, l), pl = __shfl_sync(kAll, w, l);
            if (same >> l & 1u) {
                sum += sl;
                p = a.renorm ? p + pl : pl;
            }
        }
    }
    if (first) out[id] = from_f32<T>(sum - p * dot);
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
