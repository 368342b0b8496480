// experts.cu -- the experts' products on rows sorted by expert: one block-
// diagonal sparse x dense product and its two gradients.  Rows offsets[e] ..
// offsets[e + 1] - 1 belong to expert e with weights W[e] (N x K):
//   forward   ys[p]  = W[e] xs[p]                 D = W   . xs^T   (N x rows)
//   dx        dxs[p] = W[e]^T dys[p]              D = W^T . dys^T  (K x rows)
//   dw        dW[e]  = sum_p dys[p] xs[p]^T       D = dys^T . xs   (N x K)
// One persistent warp-specialised tcgen05 kernel runs all three.  For the row
// products the weights are the MMA's M operand (128 features) and an expert's
// rows its N operand, because N may be any multiple of 16: an expert with one
// row costs one MMA of N = 16 and one with 1000 rows four of N = 256, and no
// tile of rows is padded to 128.  Rows past the expert's last one fall into
// columns of D that are not stored.  For dw the rows are the depth: the tail of
// the last 64-row block belongs to other experts and is overwritten with zeros
// in shared memory before the MMA reads it (their values may be infinite, so
// multiplying by zero would not do).
// The sums are fp32 in TMEM, rounded once to the operands' type.
//
// Roles per CTA: warp 0 loads A, warp 1 loads B (TMA, 128-byte swizzle, one
// ring of stages of 64 depth), one thread of warp 2 issues the MMAs, warps 4-7
// store D (two accumulators of 256 TMEM columns, so a unit's epilogue overlaps
// the next unit's MMAs), warp 3 writes the zero rows of dropped choices.  The
// host knows no row counts: every role walks the work units by itself, 32
// experts' offsets at a time.
#include "internal.h"
#include "rowvec.cuh"
#include "sm103.cuh"

namespace spmm {
namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kDepth = 64;       // contraction per stage: 128 bytes, one swizzle row
constexpr int kMaxTile = 256;    // columns of D per unit
constexpr int kABytes = 128 * 128;
constexpr int kStageOut = 4096;  // per epilogue warp

struct ExpertArgs {
    const int32_t* offsets;
    int32_t E, R;
    int32_t m, n;          // rows and columns of D per expert (row products: n unused)
    int32_t depth;         // contraction (dw: the expert's rows)
    int32_t m_tiles, n_tiles;
    void* out;
    int64_t ldo, lde;
    int32_t bf16;
    int* err;
    uint64_t timeout_ns;
};

// A work unit: D rows m0.. and columns n0.. (row products: rows p0 + n0 ..) of
// expert e, `nt` columns computed and `live` of them stored, `steps` stages.
struct Unit {
    int e, p0, cnt, m0, n0, nt, live, steps;
};

// Maps unit numbers to units.  Called by whole warps; unit numbers must not
// decrease.  Row products: an expert with c rows has ceil(c / 256) row tiles of
// nearly equal size times m_tiles units, row tiles fastest, so that units in
// flight together share weights.  dw: m_tiles x n_tiles units per expert.
template <int CG, bool DW>
struct Walk {
    const ExpertArgs& a;
    int lane, e0 = 0, base = 0, start = 0, cnt = 0, incl = 0;
    __device__ Walk(const ExpertArgs& args, int l) : a(args), lane(l) {
        if (!DW) window();
    }
    __device__ void window() {
        const int e = e0 + lane;
        start = e < a.E ? __ldg(a.offsets + e) : 0;
        cnt = e < a.E ? __ldg(a.offsets + e + 1) - start : 0;
        incl = (cnt + kMaxTile - 1) / kMaxTile * a.m_tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
    }
    __device__ bool find(int u, Unit& w) {
        if (DW) {
            const int per = a.m_tiles * a.n_tiles;
            if (u >= a.E * per) return false;
            w.e = u / per;
            const int i = u - w.e * per, mt = i / a.n_tiles;
            w.p0 = __ldg(a.offsets + w.e);
            w.cnt = __ldg(a.offsets + w.e + 1) - w.p0;
            w.m0 = mt * 128 * CG;
            w.n0 = (i - mt * a.n_tiles) * kMaxTile;
            w.live = min(kMaxTile, a.n - w.n0);
            w.nt = (w.live + 16 * CG - 1) / (16 * CG) * (16 * CG);
            w.steps = (w.cnt + kDepth - 1) / kDepth;
            return true;
        }
        while (true) {
            const int total = __shfl_sync(0xffffffffu, incl, 31);
            if (u - base < total) break;
            base += total;
            e0 += 32;
            if (e0 >= a.E) return false;
            window();
        }
        const int l = __ffs(__ballot_sync(0xffffffffu, u - base < incl)) - 1;
        w.e = e0 + l;
        w.p0 = __shfl_sync(0xffffffffu, start, l);
        w.cnt = __shfl_sync(0xffffffffu, cnt, l);
        const int tiles = (w.cnt + kMaxTile - 1) / kMaxTile;
        const int i = u - base - (__shfl_sync(0xffffffffu, incl, l) - tiles * a.m_tiles);
        const int mt = i / tiles, nt = i - mt * tiles;
        const int size = ((w.cnt + tiles - 1) / tiles + 16 * CG - 1) / (16 * CG) * (16 * CG);
        w.m0 = mt * 128 * CG;
        w.n0 = nt * size;
        w.live = max(0, min(size, w.cnt - w.n0));
        w.nt = size;
        w.steps = (a.depth + kDepth - 1) / kDepth;
        return true;
    }
};

template <int CG>
struct Ring {
    static constexpr int kBBytes = kMaxTile / CG * 128;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = CG == 1 ? 4 : 6;
    static constexpr int kBars = 2 * kStages + 5;
    static constexpr int kSmem = 1024 + kStages * kStage + 4 * kStageOut + kBars * 8 + 16;
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return rows::Pair<T>::pack(a, b);
}

// D columns [c, c + 32) of this warp's 32 TMEM lanes.
__device__ __forceinline__ void load32(uint32_t t, float (&v)[32]) {
    uint32_t r0[16], r1[16];
    tmem_ld16(t, r0);
    tmem_ld16(t + 16, r1);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = __uint_as_float(r0[i]);
        v[16 + i] = __uint_as_float(r1[i]);
    }
}

// Row products: lane = feature, column = row of the expert.  Every column is
// stored as 32 consecutive features by the warp.
template <typename T>
__device__ __forceinline__ void store_rows(const ExpertArgs& a, const Unit& w, uint32_t t, int feature) {
    T* out = static_cast<T*>(a.out) + static_cast<int64_t>(w.p0 + w.n0) * a.ldo + feature;
    const bool in = feature < a.m;
    for (int c = 0; c < w.live; c += 32) {
        float v[32];
        load32(t + c, v);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (in && c + i < w.live) out[(c + i) * a.ldo] = rows::from_f32<T>(v[i]);
    }
}

// dw: lane = row of dW, columns contiguous.  64 columns of the warp's 32 rows
// are staged in shared memory (16-byte units XOR-swizzled by row) and leave as
// 128-byte row segments.
template <typename T>
__device__ __forceinline__ void store_dw(const ExpertArgs& a, const Unit& w, uint32_t t, bool zero, int row0, int lane,
                                         uint32_t stage) {
    T* out = static_cast<T*>(a.out) + w.e * a.lde + w.n0;
    for (int c = 0; c < w.live; c += 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[32];
            if (zero) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
            } else {
                load32(t + c + 32 * h, v);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint4 p;
                p.x = pack2<T>(v[8 * u], v[8 * u + 1]);
                p.y = pack2<T>(v[8 * u + 2], v[8 * u + 3]);
                p.z = pack2<T>(v[8 * u + 4], v[8 * u + 5]);
                p.w = pack2<T>(v[8 * u + 6], v[8 * u + 7]);
                st_shared_v4(stage + lane * 128 + (((4 * h + u) ^ (lane & 7)) << 4), p);
            }
        }
        __syncwarp();
        const int u = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            uint4 p;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(p.x), "=r"(p.y), "=r"(p.z), "=r"(p.w)
                         : "r"(stage + r * 128 + ((u ^ (r & 7)) << 4))
                         : "memory");
            // columns come in groups of 8 (K % 8 == 0), so a group is stored whole or not at all
            if (row0 + r < a.m && c + 8 * u < w.live)
                *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row0 + r) * a.ldo + c + 8 * u) = p;
        }
        __syncwarp();
    }
}

// AMN / BMN: the operand's contiguous direction is D's row / column (else the
// depth).  BMN is dw.
template <int CG, bool AMN, bool BMN>
__global__ void __launch_bounds__(kThreads, 1)
    experts_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmB16, const ExpertArgs a) {
    using G = Ring<CG>;
    constexpr bool DW = BMN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    const uint32_t out0 = s0 + G::kStages * G::kStage;
    const uint32_t bar0 = out0 + 4 * kStageOut;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + G::kStages * G::kStage + 4 * kStageOut + 8 * G::kBars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (G::kStages + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * G::kStages + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * G::kStages + 2 + b); };
    const uint32_t done_bar = bar0 + 8u * (2 * G::kStages + 4);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int group = blockIdx.x, groups = gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(full_bar(s), 2);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), 4);
        }
        mbar_init(done_bar, 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) tma_prefetch_desc(&tmA);
    if (warp == 1 && lane == 0) tma_prefetch_desc(&tmB);
    if (warp == 2) {
        tmem_alloc(smem_u32(tslot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    Walk<CG, DW> walk(a, lane);
    Unit w;

    if (warp < 2) {
        // ------------------------------------------------ producers: A (warp 0), B (warp 1)
        int s = 0, armed = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = group; ok && walk.find(u, w); u += groups) {
            const int nb = w.nt / CG;
            for (int k = 0; k < w.steps; ++k) {
                if (!mbar_wait(empty_bar(s), ph ^ 1u, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const uint32_t st = s0 + s * G::kStage, bar = full_bar(s);
                    const int d0 = k * kDepth;
                    if (warp == 0) {
                        mbar_arrive_expect_tx(bar, kABytes);
                        if (DW) {
                            tma_load_2d(st, &tmA, bar, w.m0, w.p0 + d0);
                            tma_load_2d(st + kABytes / 2, &tmA, bar, w.m0 + 64, w.p0 + d0);
                        } else if (AMN) {
                            tma_load_3d(st, &tmA, bar, w.m0, d0, w.e);
                            tma_load_3d(st + kABytes / 2, &tmA, bar, w.m0 + 64, d0, w.e);
                        } else {
                            tma_load_3d(st, &tmA, bar, d0, w.m0, w.e);
                        }
                    } else {
                        const uint32_t sb = st + kABytes;
                        if (DW) {
                            const int boxes = (nb + 63) / 64;
                            mbar_arrive_expect_tx(bar, boxes * 8192);
                            for (int i = 0; i < boxes; ++i)
                                tma_load_2d(sb + i * 8192, &tmB, bar, w.n0 + 64 * i, w.p0 + d0);
                        } else {
                            mbar_arrive_expect_tx(bar, nb * 128);
                            const int row = w.p0 + w.n0;
                            int r = 0;
                            for (; r + 64 <= nb; r += 64) tma_load_2d(sb + r * 128, &tmB, bar, d0, row + r);
                            for (; r < nb; r += 16) tma_load_2d(sb + r * 128, &tmB16, bar, d0, row + r);
                        }
                    }
                }
                if (armed < G::kStages) ++armed;
                if (++s == G::kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // Leave no copy in flight: wait for the last phase armed on each slot.
        for (int i = 0; i < armed; ++i) {
            int idx = s - 1 - i;
            uint32_t par = ph;
            if (idx < 0) {
                idx += G::kStages;
                par ^= 1u;
            }
            mbar_wait(full_bar(idx), par, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT);
        }
    } else if (warp == 2) {
        // ------------------------------------------------ MMA issuer
        // K-major operand: +32 bytes per 16 of depth inside the swizzled row.
        // MN-major operand: chunks of 64 columns 8 KB apart, +16 rows per 16.
        const uint64_t adesc0 = AMN ? smem_desc(s0, 8192u, 1024u, SWZ_128B) : smem_desc(s0, 16u, 1024u, SWZ_128B);
        const uint64_t bdesc0 = BMN ? smem_desc(s0 + kABytes, 8192u, 1024u, SWZ_128B)
                                    : smem_desc(s0 + kABytes, 16u, 1024u, SWZ_128B);
        constexpr uint32_t kAStep = AMN ? 128 : 2, kBStep = BMN ? 128 : 2;
        int s = 0, acc = 0;
        uint32_t ph = 0, aph = 0;
        bool ok = true;
        for (int u = group; ok && walk.find(u, w); u += groups) {
            if (w.steps == 0) continue;
            if (!mbar_wait(acce_bar(acc), aph ^ 1u, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) break;
            tc_fence_after();
            const uint32_t d = tmem + static_cast<uint32_t>(acc * kMaxTile);
            const uint32_t idesc = idesc_f16(128 * CG, w.nt, a.bf16 != 0, AMN, BMN, false);
            for (int k = 0; k < w.steps; ++k) {
                if (!mbar_wait(full_bar(s), ph, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                int sub = 4;  // MMAs of 16 depth; TMA zero-filled what lies past a row product's depth
                if (DW) {
                    const int valid = w.cnt - k * kDepth;
                    if (valid < kDepth) {
                        sub = (valid + 15) / 16;
                        if (valid & 15) {
                            // rows of the next expert in the last 16: both operands become zero
                            const int chunks = 2 + (w.nt / CG + 63) / 64;
                            const int units = (sub * 16 - valid) * 8;
                            for (int c = 0; c < chunks; ++c)
                                for (int i = lane; i < units; i += 32)
                                    st_shared_v4(s0 + s * G::kStage + c * 8192 + valid * 128 + i * 16,
                                                 make_uint4(0, 0, 0, 0));
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                }
                if (lane == 0) {
                    const uint64_t so = static_cast<uint64_t>(static_cast<uint32_t>(s) * (G::kStage >> 4));
                    for (int kk = 0; kk < sub; ++kk)
                        mma_f16(d, adesc0 + so + kAStep * kk, bdesc0 + so + kBStep * kk, idesc, (k | kk) != 0 ? 1u : 0u);
                    mma_commit(empty_bar(s));
                }
                __syncwarp();
                if (++s == G::kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (lane == 0) mma_commit(accf_bar(acc));
            __syncwarp();
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
        if (lane == 0) mma_commit(done_bar);
        __syncwarp();
        mbar_wait(done_bar, 0, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT);
    } else if (warp == 3) {
        // ------------------------------------------------ zero rows of dropped choices
        if (!DW) {
            for (int64_t p = __ldg(a.offsets + a.E) + static_cast<int64_t>(blockIdx.x); p < a.R; p += gridDim.x) {
                uint4* row = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + p * a.ldo);
                for (int c = lane; c < a.m / 8; c += 32) row[c] = make_uint4(0, 0, 0, 0);
            }
        }
    } else {
        // ------------------------------------------------ epilogue
        const int q = warp & 3;  // TMEM lane quarter
        const uint32_t stage = out0 + q * kStageOut;
        int acc = 0;
        uint32_t aph = 0;
        for (int u = group; walk.find(u, w); u += groups) {
            const int row0 = w.m0 + 32 * q;
            const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kMaxTile);
            if (w.steps > 0) {
                if (!mbar_wait(accf_bar(acc), aph, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) break;
                tc_fence_after();
            }
            if (DW) {
                if (a.bf16)
                    store_dw<__nv_bfloat16>(a, w, t, w.steps == 0, row0, lane, stage);
                else
                    store_dw<__half>(a, w, t, w.steps == 0, row0, lane, stage);
            } else if (a.bf16) {
                store_rows<__nv_bfloat16>(a, w, t, row0 + lane);
            } else {
                store_rows<__half>(a, w, t, row0 + lane);
            }
            if (w.steps == 0) continue;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce_bar(acc));
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

bool weights_map(CUtensorMap* map, int32_t dtype, const void* W, int64_t ldw, int64_t lde, int64_t N, int64_t K,
                 int64_t E, uint32_t box_rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
    const uint64_t strides[2] = {static_cast<uint64_t>(ldw) * 2, static_cast<uint64_t>(lde) * 2};
    const uint32_t box[3] = {kDepth, box_rows, 1};
    return encode_tmap_3d(map, half_type(dtype), W, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool rows_map(CUtensorMap* map, int32_t dtype, const void* p, int64_t ld, int64_t R, int64_t n, uint32_t box_rows) {
    return encode_tmap_2d(map, half_type(dtype), p, static_cast<uint64_t>(n), static_cast<uint64_t>(R),
                          static_cast<uint64_t>(ld) * 2, kDepth, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int CG, bool AMN, bool BMN>
spmm_status launch(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmB16, const ExpertArgs& a,
                   int64_t units, const DeviceInfo* dev, cudaStream_t s) {
    if (units >= (int64_t(1) << 31) - dev->sms) return SPMM_ERR_UNSUPPORTED;
    const auto kern = experts_kernel<CG, AMN, BMN>;
    const int slot = kSlotExperts + (BMN ? 2 : AMN ? 1 : 0);
    if (!set_smem_attr_once(reinterpret_cast<const void*>(kern), Ring<CG>::kSmem, slot)) return SPMM_ERR_CUDA;
    const int grid = static_cast<int>(units < dev->sms ? units : dev->sms);
    trace_begin(SPMM_KERNEL_EXPERTS, s);
    kern<<<grid, kThreads, Ring<CG>::kSmem, s>>>(tmA, tmB, tmB16, a);
    const cudaError_t e = cudaGetLastError();
    trace_end(SPMM_KERNEL_EXPERTS, s);
    return cuda_status(e);
}

}  // namespace

spmm_status launch_experts_rows(const spmm_route_t* R, const void* rows, int64_t ldr, const void* W, int64_t ldw,
                                int64_t lde, int64_t N, int64_t K, bool transposed, int32_t dtype, void* out,
                                int64_t ldo, cudaStream_t s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return SPMM_ERR_CUDA;
    const int64_t n = R->T * R->k, E = R->n_keys;
    ExpertArgs a{};
    a.offsets = R->offsets;
    a.E = static_cast<int32_t>(E);
    a.R = static_cast<int32_t>(n);
    a.m = static_cast<int32_t>(transposed ? K : N);
    a.depth = static_cast<int32_t>(transposed ? N : K);
    a.out = out;
    a.ldo = ldo;
    a.bf16 = dtype == SPMM_BF16;
    a.err = dev->err;
    a.timeout_ns = kWaitTimeoutNs;
    CUtensorMap tmA, tmB, tmB16;
    if (!weights_map(&tmA, dtype, W, ldw, lde, N, K, E, transposed ? kDepth : 128) ||
        !rows_map(&tmB, dtype, rows, ldr, n, a.depth, 64) || !rows_map(&tmB16, dtype, rows, ldr, n, a.depth, 16))
        return SPMM_ERR_CUDA;
    a.m_tiles = (a.m + 127) / 128;
    // at most this many units: one partial row tile per expert with rows
    const int64_t units = (n / kMaxTile + (n < E ? n : E)) * a.m_tiles;
    return transposed ? launch<1, true, false>(tmA, tmB, tmB16, a, units, dev, s)
                      : launch<1, false, false>(tmA, tmB, tmB16, a, units, dev, s);
}

spmm_status launch_experts_dw(const spmm_route_t* R, const void* dys, int64_t ldd, const void* xs, int64_t ldx,
                              int64_t N, int64_t K, int32_t dtype, void* dW, int64_t ldw, int64_t lde, cudaStream_t s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return SPMM_ERR_CUDA;
    const int64_t n = R->T * R->k;
    ExpertArgs a{};
    a.offsets = R->offsets;
    a.E = static_cast<int32_t>(R->n_keys);
    a.R = static_cast<int32_t>(n);
    a.m = static_cast<int32_t>(N);
    a.n = static_cast<int32_t>(K);
    a.out = dW;
    a.ldo = ldw;
    a.lde = lde;
    a.bf16 = dtype == SPMM_BF16;
    a.err = dev->err;
    a.timeout_ns = kWaitTimeoutNs;
    a.m_tiles = (a.m + 127) / 128;
    a.n_tiles = (a.n + kMaxTile - 1) / kMaxTile;
    CUtensorMap tmA, tmB;
    // without rows every gradient is zero and no operand is read; the maps then cover the output's memory
    if (!rows_map(&tmA, dtype, n ? dys : dW, n ? ldd : ldw, n ? n : 1, n ? N : K, kDepth) ||
        !rows_map(&tmB, dtype, n ? xs : dW, n ? ldx : ldw, n ? n : 1, K, kDepth))
        return SPMM_ERR_CUDA;
    return launch<1, true, true>(tmA, tmB, tmB, a, static_cast<int64_t>(a.E) * a.m_tiles * a.n_tiles, dev, s);
}

}  // namespace spmm
