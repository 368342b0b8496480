// experts.cu -- the experts' products on rows sorted by expert: one block-
// diagonal sparse x dense product and its two gradients.  Rows offsets[e] ..
// offsets[e + 1] - 1 belong to expert e with weights W[e] (N x K):
//   forward   ys[p]  = W[e] xs[p]                 D = W   . xs^T   (N x rows)
//   dx        dxs[p] = W[e]^T dys[p]              D = W^T . dys^T  (K x rows)
//   dw        dW[e]  = sum_p dys[p] xs[p]^T       D = dys^T . xs   (N x K)
// One persistent warp-specialised tcgen05 kernel runs all three, on CTA pairs
// (M = 256) where D has more than 128 rows.  For the row products the weights are
// the MMA's M operand and an expert's rows its N operand, because N may be any
// multiple of 16 (32 for a pair): an expert with one row costs an MMA of N = 32
// per 256 features and one with 1000 rows four of N = 256, and no tile of rows is
// padded to 128.  Rows past the expert's last one fall into columns of D that are
// not stored.  For dw the rows are the depth: the tail of the last 64-row block
// belongs to other experts and is overwritten with zeros in shared memory before
// the MMA reads it (their values may be infinite, so multiplying by zero would
// not do).
// Why pairs: a 128 x 256 tile of one CTA loads 48 KB per 64 of depth (520 clk of
// MMA), 92 B/clk, and L2 gives an SM about 70; a pair's CTA loads 32 KB.  One
// CTA 1160 TFLOP/s, a pair 1320 on a ragged prompt batch (32768 rows, 2048 x
// 4096), 1450 with the steps below.  What bounds it now: with 1024 rows per
// expert the power limit (352 us sustained where cuBLAS's batched product takes
// 341 us), with few rows reading the weights from HBM (6.8-7.6 TB/s), between
// them the producers' and the issuing thread's instructions per step.
// The sums are fp32 in TMEM, rounded once to the operands' type.
//
// Roles per CTA: warps 0, 1, 12 and 13 load A and B (TMA, 128-byte swizzle, one
// ring of stages of 64 depth), one thread of warp 2 issues the MMAs, warps 4-11
// store D (two accumulators of 256 TMEM columns, so a unit's epilogue overlaps
// the next unit's MMAs).  The host knows no row counts: warp 3 finds this CTA's
// work units, 32 experts' offsets at a time, and announces them to the other
// warps through a ring of four (a search per role cost every role its latency
// per unit); at the end it writes the zero rows of dropped choices.
#include "internal.h"
#include "rowvec.cuh"
#include "sm103_more.cuh"

namespace spmm {
namespace {

using namespace ptx;

constexpr int kEpiWarps = 8;  // two per TMEM lane quarter, half of the columns each
constexpr int kMoreProducers = 4 + kEpiWarps;  // first warp of the second pair of producers
constexpr int kThreads = 32 * (kMoreProducers + 2);
constexpr int kDepth = 64;  // contraction per stage: 128 bytes, one swizzle row
constexpr int kABytes = 128 * 128;
constexpr int kSmemMax = 232448;  // 227 KB, the most a CTA can have
constexpr int kUnits = 4;         // work units announced ahead
// A wait may span a unit, and at the end the units announced ahead of it, and a
// unit has as many steps as its depth has blocks of 64 (dw: the rows of an
// expert).  So the limit of a wait grows with the most steps that a unit can have:
// 2 us for each, where a step takes 0.3 us and, with every SM streaming from HBM,
// 0.7.  (At 2 s flat, dw of 8 x 8 over 400 million rows, 0.33 us a step, gave up.)
constexpr uint64_t kStepLimitNs = 2000;
constexpr uint64_t wait_limit_ns(int64_t most_depth) {
    const uint64_t steps = (static_cast<uint64_t>(most_depth) + kDepth - 1) / kDepth;
    return kWaitTimeoutNs + steps * (kUnits + 1) * kStepLimitNs;
}
// Variants by size, all on averages that the host knows.
// Row tiles of 64 instead of 256 up to this many rows per expert: nine stages fit
// instead of six (64 tokens x 8 of 128 experts, 1536 x 4096: 226 us against 240).
constexpr int kFewRows = 16;
constexpr int kVecMost = 16;   // rows in all up to which the forward product runs on CUDA cores
constexpr int kDwFewRows = 4;  // rows per expert up to which dw runs on CUDA cores

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

// Tensor maps of B.  Row products load an expert's rows in boxes of 128, 64, 32
// and 16 rows (box_of); dw uses the first map for its 64 x 64 boxes.
struct BMaps {
    CUtensorMap m[4];
};
// The next box for `rest` rows (a multiple of 16): at most two boxes and 16
// unused rows per 128.  Boxes of exactly the rows needed (64 and 16) took 207 us
// where this takes 171 us (448 rows per expert): every box costs about as
// much as 32 rows.
__host__ __device__ constexpr int box_of(int rest) { return rest > 96 ? 0 : rest > 48 ? 1 : rest > 16 ? 2 : 3; }
__host__ __device__ constexpr int boxed_rows(int nb) {
    int n = 0;
    while (n < nb) n += 128 >> box_of(nb - n);
    return n;
}

// A work unit: D rows m0.. and columns n0.. (row products: rows p0 + n0 ..) of
// expert e, `nt` columns computed and `live` of them stored, `steps` stages.
struct Unit {
    int e, p0, cnt, m0, n0, nt, live, steps;
};

// Maps unit numbers to units.  Called by whole warps; unit numbers must not
// decrease.  Row products: an expert with c rows has ceil(c / 256) row tiles
// times m_tiles units, two tiles of equal size or more of 256 and a rest (320
// rows: 164 us as 160 + 160, 177 us as 256 + 64, which both read the weights at
// full length; a prompt batch of ragged experts, sustained: 374 us with full
// tiles, 380 us with equal ones); dw has n_tiles x m_tiles units per
// expert.  Inside an expert units go in groups of kGroup column tiles, column
// tiles fastest, so that the units in flight together (76 pairs) form a compact
// patch of D and share their operands in L2: with column tiles fastest over the
// whole of a 32768-row expert its rows came from HBM once per row tile of W.
constexpr int kGroup = 8;

// Tile i of m_tiles x n_tiles in that order.
__device__ __forceinline__ void tile_of(int i, int m_tiles, int n_tiles, int& mt, int& nt) {
    const int per = kGroup * m_tiles, g = i / per, rest = i - g * per;
    const int width = min(kGroup, n_tiles - g * kGroup);
    mt = rest / width;
    nt = g * kGroup + rest - mt * width;
}

template <int CG, int TILE, bool DW>
struct Walk {
    const ExpertArgs& a;
    int lane, e0 = 0, base = 0, start = 0, cnt = 0, incl = 0;
    __device__ Walk(const ExpertArgs& args, int l) : a(args), lane(l) {
        if (!DW) window();
    }
    __device__ void window() {
        const int e = e0 + lane;
        start = e < a.E ? a.offsets[e] : 0;
        cnt = e < a.E ? a.offsets[e + 1] - start : 0;
        incl = (cnt + TILE - 1) / TILE * a.m_tiles;
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
            int mt, nt;
            tile_of(u - w.e * per, a.m_tiles, a.n_tiles, mt, nt);
            w.p0 = a.offsets[w.e];
            w.cnt = a.offsets[w.e + 1] - w.p0;
            w.m0 = mt * 128 * CG;
            w.n0 = nt * TILE;
            w.live = min(TILE, a.n - w.n0);
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
        const int tiles = (w.cnt + TILE - 1) / TILE;
        const int i = u - base - (__shfl_sync(0xffffffffu, incl, l) - tiles * a.m_tiles);
        int mt, nt;
        tile_of(i, a.m_tiles, tiles, mt, nt);
        const int even = ((w.cnt + tiles - 1) / tiles + 16 * CG - 1) / (16 * CG) * (16 * CG);
        const int size = tiles > 2 ? TILE : even;
        w.m0 = mt * 128 * CG;
        w.n0 = nt * size;
        w.live = min(size, w.cnt - w.n0);
        w.nt = (w.live + 16 * CG - 1) / (16 * CG) * (16 * CG);
        w.steps = (a.depth + kDepth - 1) / kDepth;
        return true;
    }
};

// Shared memory: the ring of stages, as deep as fits, two staging buffers per
// epilogue warp (32 x 32 results of a row product, 32 x 64 of dw), barriers, units.
template <int CG, int TILE, bool DW>
struct Ring {
    static constexpr int kBBytes = TILE / CG * 128;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kBox = DW ? 4096 : 2048;  // one staging buffer
    static constexpr int kOut = 2 * kBox;
    static constexpr int kStages = (kSmemMax - 1024 - kEpiWarps * kOut - 1536) / kStage;
    static constexpr int kBars = 4 * kStages + 5 + 2 * kUnits;
    static constexpr int kBarOff = kStages * kStage + kEpiWarps * kOut;
    static constexpr int kUnitOff = kBarOff + kBars * 8 + 16;
    static constexpr int kSmem = 1024 + kUnitOff + kUnits * static_cast<int>(sizeof(Unit));
    static_assert(kSmem <= kSmemMax && kStages <= 16, "fits an SM; barrier phases fit a word");
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b) {
    return rows::Pair<T>::pack(__uint_as_float(a), __uint_as_float(b));
}

// Row products: TMEM lane = feature, column = row of the expert.  Blocks of 8
// features x 8 rows are transposed on their way to shared memory (32 rows x 32
// features, 16-byte units XOR-swizzled by row).  A box of 32 live rows leaves as
// one TMA store; the last rows of a tile, whose successors belong to another
// expert, in 16-byte pieces.
template <typename T>
__device__ __forceinline__ void store_rows(const ExpertArgs& a, const CUtensorMap* tmOut, const Unit& w, uint32_t t,
                                           int c0, int c1, int row0, int lane, uint32_t buffers, int& odd) {
    T* out = static_cast<T*>(a.out) + static_cast<int64_t>(w.p0 + w.n0) * a.ldo;
    const int unit = lane & 3, feature = row0 + 8 * unit;
    for (int c = c0; c < c1; c += 32, odd ^= 1) {
        const uint32_t stage = buffers + odd * 2048;
        const uint32_t put = stage + (lane & 7) * 64 + (((lane >> 3) ^ ((lane & 7) >> 1)) << 4);
        uint32_t lo[16], hi[16];
        __syncwarp();  // TMEM loads are .aligned; the warp comes from a spinning wait or one thread's store
        tmem_ld_16x32(t + c, lo);
        tmem_ld_16x32(t + (16u << 16) + c, hi);
        tmem_ld_wait();
        if (lane == 0) bulk_wait_read<1>();  // the store before last has read this buffer
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b)  // rows 8 b .. 8 b + 7
            stmatrix_x4_trans(put + b * 512, pack2<T>(lo[4 * b], lo[4 * b + 1]), pack2<T>(lo[4 * b + 2], lo[4 * b + 3]),
                              pack2<T>(hi[4 * b], hi[4 * b + 1]), pack2<T>(hi[4 * b + 2], hi[4 * b + 3]));
        if (c + 32 <= c1) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (row0 < a.m) tma_store_2d(tmOut, stage, row0, w.p0 + w.n0 + c);
                bulk_commit();
            }
            continue;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2);
            const uint4 p = ld_shared_v4(stage + r * 64 + ((unit ^ ((r >> 1) & 3)) << 4));
            // features come in groups of 8 (N % 8 == 0), so a group is stored whole or not at all
            if (feature < a.m && c + r < c1) __stcs(reinterpret_cast<uint4*>(out + (c + r) * a.ldo + feature), p);
        }
        if (lane == 0) bulk_commit();  // an empty group: one per use of a buffer
        __syncwarp();
    }
}

// dw: TMEM lane = row of dW, columns contiguous.  64 columns of the warp's 32
// rows are staged in shared memory (16-byte units XOR-swizzled by row) and leave
// as one TMA store, which drops what lies past dW's edges.
template <typename T>
__device__ __forceinline__ void store_dw(const ExpertArgs& a, const CUtensorMap* tmOut, const Unit& w, uint32_t t,
                                         int c0, int c1, int row0, int lane, uint32_t buffers, int& odd) {
    for (int c = c0; c < c1; c += 64, odd ^= 1) {
        const uint32_t stage = buffers + odd * 4096;
        uint32_t v[4][16];
        __syncwarp();  // as in store_rows
        if (w.steps == 0) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i) v[h][i] = 0u;
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) tmem_ld16(t + c + 16 * h, v[h]);
            tmem_ld_wait();
        }
        if (lane == 0) bulk_wait_read<1>();  // the store before last has read this buffer
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t* f = &v[u >> 1][8 * (u & 1)];
            st_shared_v4(stage + lane * 128 + ((u ^ (lane & 7)) << 4),
                         make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                                    pack2<T>(f[6], f[7])));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (row0 < a.m) tma_store_3d(tmOut, stage, w.n0 + c, row0, w.e);
            bulk_commit();
        }
    }
}

// dw: rows [valid, end) of a stage's chunks (64 columns each, 64 rows of 128
// bytes) become zero.  Called by a whole warp.
__device__ __forceinline__ void clear_tail(uint32_t stage, int valid, int end, int chunks, int lane) {
    for (int c = 0; c < chunks; ++c)
        for (int i = lane; i < (end - valid) * 8; i += 32)
            st_shared_v4(stage + c * 8192 + valid * 128 + i * 16, make_uint4(0, 0, 0, 0));
    fence_proxy_async_smem();
    __syncwarp();
}

// One CTA (CG = 1) or a pair (CG = 2) per MMA.
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                    uint32_t idesc, uint32_t acc, uint32_t issue) {
    if (CG == 2)
        mma_f16_pair(d, a_lo, a_hi, b_lo, b_hi, idesc, acc, issue);
    else
        mma_f16_single(d, a_lo, a_hi, b_lo, b_hi, idesc, acc, issue);
}
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (CG == 2)
        mma_commit_pair(bar);
    else
        mma_commit(bar);
}
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
    if (CG == 2)
        tma_load_2d_pair(dst, m, bar, c0, c1);
    else
        tma_load_2d(dst, m, bar, c0, c1);
}
template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
    if (CG == 2)
        tma_load_3d_pair(dst, m, bar, c0, c1, c2);
    else
        tma_load_3d(dst, m, bar, c0, c1, c2);
}
template <int CG>
__device__ __forceinline__ void sync_all() {
    if (CG == 2)
        cluster_sync_all();
    else
        __syncthreads();
}

// AMN / BMN: the operand's contiguous direction is D's row / column (else the
// depth).  BMN is dw.
template <int CG, int TILE, bool AMN, bool BMN>
__global__ void __launch_bounds__(kThreads, 1)
    experts_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ BMaps tmB,
                   const __grid_constant__ CUtensorMap tmOut, const ExpertArgs a) {
    constexpr bool DW = BMN;
    using G = Ring<CG, TILE, DW>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    const uint32_t out0 = s0 + G::kStages * G::kStage;
    const uint32_t bar0 = s0 + G::kBarOff;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + G::kBarOff + 8 * G::kBars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (G::kStages + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * G::kStages + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * G::kStages + 2 + b); };
    const uint32_t done_bar = bar0 + 8u * (2 * G::kStages + 4);
    auto tail_bar = [&](int s) { return done_bar + 8u + 8u * s; };
    auto zeroed_bar = [&](int s) { return done_bar + 8u + 8u * (G::kStages + s); };
    auto unitf_bar = [&](int i) { return done_bar + 8u + 8u * (2 * G::kStages + i); };
    auto unite_bar = [&](int i) { return done_bar + 8u + 8u * (2 * G::kStages + kUnits + i); };
    Unit* ring = reinterpret_cast<Unit*>(smem + G::kUnitOff);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int group = blockIdx.x / CG, groups = gridDim.x / CG;
    const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            mbar_init(tail_bar(s), 1);
            mbar_init(zeroed_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), kEpiWarps * CG);
        }
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(unitf_bar(i), 1);
            mbar_init(unite_bar(i), kThreads / 32 - 1);  // every warp but the walking one
        }
        mbar_init(done_bar, 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) tma_prefetch_desc(&tmA);
    if (warp == 1 && lane == 0) tma_prefetch_desc(&tmB.m[0]);
    // The setup above runs beside the end of the kernel before.  TMEM is taken only after it has
    // ended (it may still want TMEM of its own) and before the next kernel may start.
    grid_dep_wait();
    if (warp == 2) {
        if (CG == 2) {
            tmem_alloc_pair(smem_u32(tslot), 2 * TILE);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tslot), 2 * TILE);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    sync_all<CG>();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    grid_dep_launch();
    Unit w;
    // the next unit for this warp; false after the last one
    int ui = 0;
    uint32_t uph = 0;
    auto next_unit = [&]() {
        if (!mbar_wait(unitf_bar(ui), uph, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) return false;
        w = ring[ui];
        __syncwarp();
        if (lane == 0) mbar_arrive(unite_bar(ui));
        if (++ui == kUnits) {
            ui = 0;
            uph ^= 1u;
        }
        return w.e >= 0;
    };

    if (warp < 2 || warp >= kMoreProducers) {
        // ------------------------------------------------ producers
        // Two pairs of warps, one for even and one for odd steps (counted over all units); in a pair one
        // warp loads A and the other B.  A TMA instruction costs its warp 100-200 clk, and a single pair
        // with two boxes per operand needed 560 clk a step where the MMAs need 520.
        const bool loads_a = (warp & 1) == 0;
        int turn = warp >= kMoreProducers;  // steps until this warp's next one, modulo 2
        int s = 0, armed = 0;
        uint32_t ph = 0;
        const uint32_t full0 = CG == 2 ? map_shared(full_bar(0), 0) : full_bar(0);
        bool ok = true;
        while (ok && next_unit()) {
            const int nb = w.nt / CG, m0 = w.m0 + 128 * rank, n0 = w.n0 + nb * rank;
            const uint32_t b_bytes = DW ? (nb + 63) / 64 * 8192 : boxed_rows(nb) * 128;
            for (int k = 0; k < w.steps; ++k, turn ^= 1) {
                if (turn == 0 && !mbar_wait(empty_bar(s), ph ^ 1u, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) {
                    ok = false;
                    break;
                }
                if (turn == 0 && lane == 0) {
                    const uint32_t st = s0 + s * G::kStage;
                    const int d0 = k * kDepth;
                    // A pair's loads all complete on rank 0's barrier.  A dw tail that rank 1 has to clear
                    // first completes on rank 1's own barrier instead.
                    const bool tail = CG == 2 && DW && ((w.cnt - d0) & 15) && w.cnt - d0 < kDepth;
                    const uint32_t own = tail && rank ? tail_bar(s) : full_bar(s);
                    const uint32_t bar = CG == 1 || tail ? own : full0 + 8u * s;
                    if (loads_a) {
                        // the one arrival of the phase, for both warps' copies (and both CTAs', unless
                        // they wait apart); copies that land before it only lower the count first
                        if (rank == 0 || tail)
                            mbar_arrive_expect_tx(own, (kABytes + b_bytes) * (tail ? 1 : CG));
                        if (DW) {
                            load_2d<CG>(st, &tmA, bar, m0, w.p0 + d0);
                            load_2d<CG>(st + kABytes / 2, &tmA, bar, m0 + 64, w.p0 + d0);
                        } else if (AMN) {
                            load_3d<CG>(st, &tmA, bar, m0, d0, w.e);
                            load_3d<CG>(st + kABytes / 2, &tmA, bar, m0 + 64, d0, w.e);
                        } else {
                            load_3d<CG>(st, &tmA, bar, d0, m0, w.e);
                        }
                    } else {
                        const uint32_t sb = st + kABytes;
                        if (DW) {
                            for (int c = 0; c < nb; c += 64)
                                load_2d<CG>(sb + c * 128, &tmB.m[0], bar, n0 + c, w.p0 + d0);
                        } else {
                            for (int r = 0; r < nb;) {
                                const int b = box_of(nb - r);
                                load_2d<CG>(sb + r * 128, &tmB.m[b], bar, d0, w.p0 + n0 + r);
                                r += 128 >> b;
                            }
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
        // Leave no copy in flight: wait for the last phase armed on each slot (rank 0 holds the
        // barriers of both CTAs' copies).
        for (int i = 0; rank == 0 && i < armed; ++i) {
            int idx = s - 1 - i;
            uint32_t par = ph;
            if (idx < 0) {
                idx += G::kStages;
                par ^= 1u;
            }
            mbar_wait(full_bar(idx), par, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT);
        }
    } else if (warp == 2 && rank == 0) {
        // ------------------------------------------------ MMA issuer
        // K-major operand: +32 bytes per 16 of depth inside the swizzled row.
        // MN-major operand: chunks of 64 columns 8 KB apart, +16 rows per 16.
        const uint64_t adesc0 = AMN ? smem_desc(s0, 8192u, 1024u, SWZ_128B) : smem_desc(s0, 16u, 1024u, SWZ_128B);
        const uint64_t bdesc0 = BMN ? smem_desc(s0 + kABytes, 8192u, 1024u, SWZ_128B)
                                    : smem_desc(s0 + kABytes, 16u, 1024u, SWZ_128B);
        constexpr uint32_t kAStep = AMN ? 128 : 2, kBStep = BMN ? 128 : 2;
        const uint32_t a_hi = static_cast<uint32_t>(adesc0 >> 32), b_hi = static_cast<uint32_t>(bdesc0 >> 32);
        const uint32_t issue = lane == 0;
        int s = 0, acc = 0;
        uint32_t ph = 0, aph = 0, zph = 0;
        bool ok = true;
        while (ok && next_unit()) {
            if (w.steps == 0) continue;
            if (!(CG == 2 ? mbar_wait_cluster(acce_bar(acc), aph ^ 1u, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)
                          : mbar_wait(acce_bar(acc), aph ^ 1u, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)))
                break;
            tc_fence_after();
            const uint32_t d = tmem + static_cast<uint32_t>(acc * TILE);
            const uint32_t idesc = idesc_f16(128 * CG, w.nt, a.bf16 != 0, AMN, BMN, false);
            // whole stages; the loop stays warp-uniform around the one issuing thread, which keeps the
            // descriptors in uniform registers
            const int whole = DW ? w.cnt / kDepth : w.steps;
            bool ready = whole > 0 && mbar_test_wait(full_bar(s), ph);
            for (int k = 0; k < whole; ++k) {
                if (!ready && !mbar_wait(full_bar(s), ph, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t so = static_cast<uint32_t>(s) * (G::kStage >> 4), empty = empty_bar(s);
                if (++s == G::kStages) {
                    s = 0;
                    ph ^= 1u;
                }
                // the next stage's test is on its way while this stage's MMAs are issued
                ready = k + 1 < whole && mbar_test_wait(full_bar(s), ph);
                const uint32_t a_lo = static_cast<uint32_t>(adesc0) + so, b_lo = static_cast<uint32_t>(bdesc0) + so;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma<CG>(d, a_lo + kAStep * kk, a_hi, b_lo + kBStep * kk, b_hi, idesc, (k | kk) != 0 ? 1u : 0u, issue);
                if (lane == 0) commit<CG>(empty);
                __syncwarp();
            }
            if (DW && ok && whole < w.steps) {
                // the tail: MMAs of 16 rows up to the expert's last, what follows it cleared
                const int valid = w.cnt - whole * kDepth, sub = (valid + 15) / 16;
                ok = mbar_wait(full_bar(s), ph, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT);
                if (valid & 15) {
                    clear_tail(s0 + s * G::kStage, valid, sub * 16, 2 + (w.nt / CG + 63) / 64, lane);
                    if (CG == 2) {
                        ok = ok && mbar_wait_cluster(zeroed_bar(s), (zph >> s) & 1u, a.timeout_ns, a.err,
                                                     SPMM_DEVERR_TIMEOUT);
                        zph ^= 1u << s;
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                if (lane == 0 && ok) {
                    const uint32_t so = static_cast<uint32_t>(s) * (G::kStage >> 4);
                    const uint32_t a_lo = static_cast<uint32_t>(adesc0) + so, b_lo = static_cast<uint32_t>(bdesc0) + so;
                    for (int kk = 0; kk < sub; ++kk)
                        mma<CG>(d, a_lo + kAStep * kk, a_hi, b_lo + kBStep * kk, b_hi, idesc,
                                (whole | kk) != 0 ? 1u : 0u, 1u);
                    commit<CG>(empty_bar(s));
                }
                if (++s == G::kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            __syncwarp();
            if (lane == 0) commit<CG>(accf_bar(acc));
            __syncwarp();
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
        if (lane == 0) commit<CG>(done_bar);
        __syncwarp();
        mbar_wait(done_bar, 0, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT);
    } else if (warp == 2) {
        // ------------------------------------------------ rank 1 of a pair: dw clears its own tails.
        // Tails of short units may be in flight together, so each slot has its own barriers.
        int s = 0;
        uint32_t ph = 0;
        while (next_unit()) {
            if (!DW) continue;
            s = (s + w.steps) % G::kStages;
            const int valid = w.cnt % kDepth;
            if ((valid & 15) == 0) continue;
            const int last = s == 0 ? G::kStages - 1 : s - 1;
            if (!mbar_wait(tail_bar(last), (ph >> last) & 1u, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) break;
            ph ^= 1u << last;
            clear_tail(s0 + last * G::kStage, valid, (valid + 15) / 16 * 16, 2 + (w.nt / CG + 63) / 64, lane);
            if (lane == 0) mbar_arrive_remote(map_shared(zeroed_bar(last), 0));
            __syncwarp();
        }
        // rank 0's last commit has arrived here: none of its arrivals is still on its way at exit
        mbar_wait(done_bar, 0, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT);
    } else if (warp == 3) {
        // ------------------------------------------------ work units, and the zero rows of dropped choices
        Walk<CG, TILE, DW> walk(a, lane);
        bool more = true;
        for (int u = group; more; u += groups) {
            more = walk.find(u, w);
            if (!more) w.e = -1;
            if (!mbar_wait(unite_bar(ui), uph ^ 1u, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) break;
            if (lane == 0) {
                ring[ui] = w;
                mbar_arrive(unitf_bar(ui));
            }
            __syncwarp();
            if (++ui == kUnits) {
                ui = 0;
                uph ^= 1u;
            }
        }
        if (!DW) {
            for (int64_t p = a.offsets[a.E] + static_cast<int64_t>(blockIdx.x); p < a.R; p += gridDim.x) {
                uint4* row = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + p * a.ldo);
                for (int c = lane; c < a.m / 8; c += 32) row[c] = make_uint4(0, 0, 0, 0);
            }
        }
    } else {  // warps 4 .. 11
        // ------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - 4) >> 2;  // TMEM lane quarter, half of the columns
        const uint32_t stage = out0 + (warp - 4) * G::kOut;
        int acc = 0;
        int odd = 0;  // the staging buffers alternate across units too: only the newest store may be unread
        uint32_t aph = 0;
        while (next_unit()) {
            const int row0 = w.m0 + 128 * rank + 32 * q;
            const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * TILE);
            if (w.steps > 0) {
                if (!mbar_wait(accf_bar(acc), aph, a.timeout_ns, a.err, SPMM_DEVERR_TIMEOUT)) break;
                tc_fence_after();
            }
            // columns past the live ones of this warp's half are computed but not stored
            const int c0 = half * (TILE / 2), c1 = min(w.live, c0 + TILE / 2);
            if (DW) {
                if (a.bf16)
                    store_dw<__nv_bfloat16>(a, &tmOut, w, t, c0, c1, row0, lane, stage, odd);
                else
                    store_dw<__half>(a, &tmOut, w, t, c0, c1, row0, lane, stage, odd);
            } else if (a.bf16) {
                store_rows<__nv_bfloat16>(a, &tmOut, w, t, c0, c1, row0, lane, stage, odd);
            } else {
                store_rows<__half>(a, &tmOut, w, t, c0, c1, row0, lane, stage, odd);
            }
            if (w.steps == 0) continue;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0)
                    mbar_arrive(acce_bar(acc));
                else
                    mbar_arrive_remote(map_shared(acce_bar(acc), 0));
            }
            __syncwarp();
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
        if (lane == 0) bulk_wait<0>();  // this warp's stores have completed
    }

    tc_fence_before();
    __syncwarp();
    sync_all<CG>();
    if (warp == 2) {
        tc_fence_after();
        if (CG == 2)
            tmem_dealloc_pair(tmem, 2 * TILE);
        else
            tmem_dealloc(tmem, 2 * TILE);
    }
}

// ---------------------------------------------------------------- a token or two
// The forward product of very few rows: dot products on CUDA cores.  A pair of
// the kernel above streams weights at 60-67 GB/s per SM whatever its depth of
// stages, and one token with 8 experts of 1536 features makes 48 pairs; here
// every warp takes two weight rows, so the read spreads over all SMs.  Measured
// (one token, 8 of 128 experts, 1536 x 4096 bf16): 20.3 us against 22.9 us, 2 of
// 16 experts, 4096 x 14336: 38 us (6.2 TB/s) against 60 us; two tokens 32 us
// against 43 us.  At four tokens the two are even, and rows that share an expert
// read its weights once per four rows here (16 tokens, 2 of 8 experts: 67 us
// against 44 us), hence the limit of 16 rows.
struct VecArgs {
    const int32_t* offsets;
    int32_t E;
    const void *xs, *W;
    int64_t ldx, ldw, lde;
    int32_t N, K;
    void* out;
    int64_t ldo;
};
constexpr int kVecWarps = 8, kVecRows = 4, kVecFeatures = 2 * kVecWarps;

// Two weight rows with C rows of xs.
template <typename T, int C>
__device__ __forceinline__ void dot_rows(const VecArgs& a, const T* w0, const T* w1, const T* x, T* out, int lane) {
    using V = rows::Vec<T, 8>;
    float acc[2][C] = {};
    // per weight row; at four CTAs per SM (64 registers) 48-52 bytes of spills are loaded, with 4 128-140
    constexpr int kFlight = 2;
    for (int k0 = lane * 8; k0 < a.K; k0 += 256 * kFlight) {
        uint4 r[2][kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int k = k0 + 256 * i;
            r[0][i] = k < a.K ? ptx::ld_global_cs(reinterpret_cast<const uint4*>(w0 + k)) : V::zero();
            r[1][i] = k < a.K ? ptx::ld_global_cs(reinterpret_cast<const uint4*>(w1 + k)) : V::zero();
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
        if (lane == 0) {
            out[c * a.ldo] = rows::from_f32<T>(acc[0][c]);
            out[c * a.ldo + 1] = rows::from_f32<T>(acc[1][c]);
        }
    }
}

// Grid (16 features, sorted place): the CTAs of an expert's first place and of
// every fourth after it take up to four of its rows, the others leave; places of
// dropped choices are zeroed.
template <typename T>
__global__ void __launch_bounds__(kVecWarps * 32, 4) experts_vec_kernel(const VecArgs a) {
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = blockIdx.y, n = (blockIdx.x * kVecWarps + warp) * 2;
    if (n >= a.N) return;  // N is even: n + 1 is a feature too
    T* out = static_cast<T*>(a.out) + p * a.ldo + n;
    if (p >= a.offsets[a.E]) {
        if (lane < 2) out[lane] = rows::from_f32<T>(0.f);
        return;
    }
    int lo = 0, hi = a.E;  // the last e with offsets[e] <= p, 32 probes at a time
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + step * lane;
        const uint32_t le = __ballot_sync(0xffffffffu, at < hi && a.offsets[at] <= p);
        lo += step * (31 - __clz(le));
        hi = min(hi, lo + step);
    }
    if ((p - a.offsets[lo]) % kVecRows) return;
    const int rows = min(kVecRows, a.offsets[lo + 1] - p);
    const T* x = static_cast<const T*>(a.xs) + p * a.ldx;
    const T* w0 = static_cast<const T*>(a.W) + lo * a.lde + n * a.ldw;
    const T* w1 = w0 + a.ldw;
    if (rows == 1)
        dot_rows<T, 1>(a, w0, w1, x, out, lane);
    else if (rows == 2)
        dot_rows<T, 2>(a, w0, w1, x, out, lane);
    else if (rows == 3)
        dot_rows<T, 3>(a, w0, w1, x, out, lane);
    else
        dot_rows<T, 4>(a, w0, w1, x, out, lane);
}

// dw of few rows per expert is a write: E N K values from a handful of rows. The
// kernel above stores tiles at 4.8 TB/s at best (an SM's loads and stores cost
// nearly their sum: 185 us with 64 rows per expert, 122 us for the same stores
// alone); here short-lived CTAs write the gradient in address order, 8 of its
// rows at a time, from sums on CUDA cores (two products per instruction).
// Measured (64 experts, 1536 x 4096, 805 MB): 107 us with a row per expert
// (7.5 TB/s) against 139 us, 134 us against 154 us with four, 184 us against
// 167 us with eight, hence the limit of four per expert on average.
struct DwArgs {
    const int32_t* offsets;
    const void *dys, *xs;
    int64_t ldd, ldx, ldw, lde;
    int32_t N, K;
    void* dW;
};
constexpr int kDwRows = 8, kDwThreads = 128, kDwDepth = 16;  // rows of dW per CTA; rows of dys staged at a time
constexpr int kDwFlight = 4;                                 // rows of xs in flight per thread

template <typename T>
__global__ void __launch_bounds__(kDwThreads, 4) experts_dw_vec_kernel(const DwArgs a) {
    using V = rows::Vec<T, 8>;
    __shared__ __align__(16) uint64_t d[kDwDepth][kDwRows];  // each value twice
    grid_dep_launch();
    grid_dep_wait();
    const int64_t e = blockIdx.y, n0 = static_cast<int64_t>(blockIdx.x) * kDwRows;
    const int32_t p0 = a.offsets[e], cnt = a.offsets[e + 1] - p0;
    const T* dys = static_cast<const T*>(a.dys) + p0 * a.ldd + n0;
    const T* xs = static_cast<const T*>(a.xs) + p0 * a.ldx;
    T* out = static_cast<T*>(a.dW) + e * a.lde + n0 * a.ldw;
    for (int k0 = 0; k0 < a.K; k0 += kDwThreads * 8) {
        const int k = k0 + threadIdx.x * 8;
        const bool in = k < a.K;
        uint64_t acc[kDwRows][4] = {};  // pairs of fp32 sums
        for (int c0 = 0; c0 < cnt; c0 += kDwDepth) {
            const int nc = min(kDwDepth, cnt - c0);
            if (k0 == 0 || cnt > kDwDepth) {  // one batch stays staged for all columns
                __syncthreads();
                if (static_cast<int>(threadIdx.x) < nc * kDwRows) {  // N % 8 == 0: every row exists
                    const int c = threadIdx.x / kDwRows, r = threadIdx.x % kDwRows;
                    const float v = rows::to_f32<T>(dys[(c0 + c) * a.ldd + r]);
                    d[c][r] = pair_f32(v, v);
                }
                __syncthreads();
            }
            if (!in) continue;
            for (int c1 = 0; c1 < nc; c1 += kDwFlight) {
                uint4 raw[kDwFlight];
#pragma unroll
                for (int i = 0; i < kDwFlight; ++i)
                    raw[i] = c1 + i < nc ? V::load(xs + (c0 + c1 + i) * a.ldx + k) : V::zero();
#pragma unroll
                for (int i = 0; i < kDwFlight; ++i) {
                    if (c1 + i >= nc) break;
                    float x[8];
                    V::unpack(raw[i], x);
                    uint64_t xx[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) xx[j] = pair_f32(x[2 * j], x[2 * j + 1]);
#pragma unroll
                    for (int r = 0; r < kDwRows; ++r)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[r][j] = fma_f32x2(d[c1 + i][r], xx[j], acc[r][j]);
                }
            }
        }
        if (!in) continue;
#pragma unroll
        for (int r = 0; r < kDwRows; ++r) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 p = unpair_f32(acc[r][j]);
                f[2 * j] = p.x;
                f[2 * j + 1] = p.y;
            }
            V::store_cs(out + r * a.ldw + k, V::pack(f));
        }
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

template <int CG, int TILE, bool AMN, bool BMN>
spmm_status launch(const CUtensorMap& tmA, const BMaps& tmB, const CUtensorMap& tmOut, const ExpertArgs& a,
                   int64_t units, const DeviceInfo* dev, cudaStream_t s) {
    if (units >= (int64_t(1) << 31) - dev->sms) return SPMM_ERR_UNSUPPORTED;
    const auto kern = experts_kernel<CG, TILE, AMN, BMN>;
    constexpr int smem = Ring<CG, TILE, BMN>::kSmem;
    constexpr int slot = kSlotExperts + (TILE < 256 ? 6 : 0) + (CG - 1) * 3 + (BMN ? 2 : AMN ? 1 : 0);
    if (!set_smem_attr_once(reinterpret_cast<const void*>(kern), smem, slot)) return SPMM_ERR_CUDA;
    const int64_t groups = units < dev->sms / CG ? units : dev->sms / CG;
    trace_begin(SPMM_KERNEL_EXPERTS, s);
    const cudaError_t e = launch_chained(kern, static_cast<unsigned>(groups * CG), kThreads, smem, CG, s, tmA, tmB,
                                         tmOut, a);
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
    if (!transposed && n <= kVecMost) {
        const VecArgs v{R->offsets, static_cast<int32_t>(E), rows, W,   ldr, ldw, lde, static_cast<int32_t>(N),
                        static_cast<int32_t>(K), out, ldo};
        const dim3 grid(static_cast<unsigned>((N + kVecFeatures - 1) / kVecFeatures), static_cast<unsigned>(n));
        trace_begin(SPMM_KERNEL_EXPERTS, s);
        const cudaError_t e = dtype == SPMM_BF16
                                  ? launch_chained(experts_vec_kernel<__nv_bfloat16>, grid, kVecWarps * 32, 0, 1, s, v)
                                  : launch_chained(experts_vec_kernel<__half>, grid, kVecWarps * 32, 0, 1, s, v);
        trace_end(SPMM_KERNEL_EXPERTS, s);
        return cuda_status(e);
    }
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
    a.timeout_ns = wait_limit_ns(a.depth);
    const bool pair = a.m > 128;
    a.m_tiles = pair ? (a.m + 255) / 256 : (a.m + 127) / 128;
    const int tile = pair && n <= E * kFewRows ? 64 : 256;
    CUtensorMap tmA, tmOut;
    BMaps tmB{};
    if (!weights_map(&tmA, dtype, W, ldw, lde, N, K, E, transposed ? kDepth : 128)) return SPMM_ERR_CUDA;
    // the boxes that a tile of an expert with at most n rows can ask for (encoding a map costs the host 1-2 us)
    const int64_t most = ((n < tile ? n : tile) + 31) / 32 * 32 / (pair ? 2 : 1);
    for (int i = box_of(static_cast<int>(most)); i < 4; ++i)
        if (!rows_map(&tmB.m[i], dtype, rows, ldr, n, a.depth, 128u >> i)) return SPMM_ERR_CUDA;
    if (!encode_tmap_2d(&tmOut, half_type(dtype), out, static_cast<uint64_t>(a.m), static_cast<uint64_t>(n),
                        static_cast<uint64_t>(ldo) * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
        return SPMM_ERR_CUDA;
    // at most this many units: one partial row tile per expert with rows
    const int64_t units = (n / tile + (n < E ? n : E)) * a.m_tiles;
    if (tile == 64)
        return transposed ? launch<2, 64, true, false>(tmA, tmB, tmOut, a, units, dev, s)
                          : launch<2, 64, false, false>(tmA, tmB, tmOut, a, units, dev, s);
    if (pair)
        return transposed ? launch<2, 256, true, false>(tmA, tmB, tmOut, a, units, dev, s)
                          : launch<2, 256, false, false>(tmA, tmB, tmOut, a, units, dev, s);
    return transposed ? launch<1, 256, true, false>(tmA, tmB, tmOut, a, units, dev, s)
                      : launch<1, 256, false, false>(tmA, tmB, tmOut, a, units, dev, s);
}

spmm_status launch_experts_dw(const spmm_route_t* R, const void* dys, int64_t ldd, const void* xs, int64_t ldx,
                              int64_t N, int64_t K, int32_t dtype, void* dW, int64_t ldw, int64_t lde, cudaStream_t s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return SPMM_ERR_CUDA;
    const int64_t n = R->T * R->k;
    if (n <= R->n_keys * kDwFewRows) {
        const DwArgs v{R->offsets, dys, xs, ldd, ldx, ldw, lde, static_cast<int32_t>(N), static_cast<int32_t>(K), dW};
        const dim3 grid(static_cast<unsigned>(N / kDwRows), static_cast<unsigned>(R->n_keys));
        trace_begin(SPMM_KERNEL_EXPERTS, s);
        const cudaError_t e = dtype == SPMM_BF16
                                  ? launch_chained(experts_dw_vec_kernel<__nv_bfloat16>, grid, kDwThreads, 0, 1, s, v)
                                  : launch_chained(experts_dw_vec_kernel<__half>, grid, kDwThreads, 0, 1, s, v);
        trace_end(SPMM_KERNEL_EXPERTS, s);
        return cuda_status(e);
    }
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
    a.timeout_ns = wait_limit_ns(n);
    const bool pair = a.m > 128;
    a.m_tiles = pair ? (a.m + 255) / 256 : (a.m + 127) / 128;
    a.n_tiles = (a.n + 255) / 256;
    CUtensorMap tmA, tmOut;
    BMaps tmB{};
    if (!weights_map(&tmOut, dtype, dW, ldw, lde, N, K, a.E, 32)) return SPMM_ERR_CUDA;
    if (!rows_map(&tmA, dtype, dys, ldd, n, N, kDepth) || !rows_map(&tmB.m[0], dtype, xs, ldx, n, K, kDepth))
        return SPMM_ERR_CUDA;
    const int64_t units = static_cast<int64_t>(a.E) * a.m_tiles * a.n_tiles;
    return pair ? launch<2, 256, true, true>(tmA, tmB, tmOut, a, units, dev, s)
                : launch<1, 256, true, true>(tmA, tmB, tmOut, a, units, dev, s);
}

}  // namespace spmm
