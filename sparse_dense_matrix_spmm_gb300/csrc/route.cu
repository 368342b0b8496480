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
#include "sm103_more.cuh"

namespace spmm {
namespace {

using namespace rows;

// ---------------------------------------------------------------- sort
// Least-significant-digit radix sort, up to 9 bits per pass, in tiles of 2048
// elements.  Inside a tile a warp owns consecutive elements and ranks them with
// one ballot per digit bit; a digit's place is the sum of the smaller digits, of
// the earlier tiles' and of the earlier warps' counts.  So the order is that of
// the input and nothing depends on the order of atomics.  By size:
//   1 tile         one CTA, one launch
//   2 .. 8 tiles   one cluster, one launch: the CTAs read each other's counts
//                  and hand the elements from pass to pass through distributed
//                  shared memory (one tile: through its own)
//   more           one launch per pass over up to kMaxCtas CTAs, and one that
//                  counts for the first pass; placing an element counts its next
//                  digit for the CTA that will read it there
// The kernels are bound by latency (launches, barriers, chains of dependent
// loads); measured in a graph with 8 choices per token and 128 keys: 16 tokens
// 3.6 us, 256 tokens 4.8 us, 1024 tokens 5.5 us (7.4 us as two launches), 16384
// tokens 11.4 us (11.8 us with loads past L1); 32768 ids over 131072 keys (two
// passes and the offsets) 21.7 us.  Elements handed on in shared memory against a
// round trip through L2: 2048 ids over 50000 keys 11.7 us against 13.7 us, 8192
// ids 15.8 us against 17.9 us, 2049 ids over 300000 keys (three passes) 15.8 us
// against 21.9 us.
// One cluster over everything, with ranks from match_any, took 56 us for 16384
// tokens (8 SMs' issue slots); 16 CTAs per cluster gained nothing over 8.
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortThreads = 512;  // one per bin
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kItems = 4;          // per thread and tile
constexpr int kTile = kSortThreads * kItems;

constexpr int kMaxCluster = 8;  // the portable limit
constexpr int kMaxCtas = 128;  // each reads every CTA's counts (256 CTAs for 524288 elements: 30 us in those reads)

struct SortArgs {
    const void* ids;
    int64_t ldi;   // row pitch of ids in elements
    int32_t wide;  // ids are 64-bit
    int32_t k, n, n_keys, passes, bits;
    int32_t chunk;  // elements per CTA, a multiple of kTile
    int32_t *order, *pos, *offsets, *keys;  // keys: the sorted keys, or null
    int32_t *keys0, *idx0, *keys1, *idx1;  // results of even and odd passes
    int32_t* table;                    // [passes][CTAs][bins] digit counts
    int* err;
};

// Key of flat index f: its id, or n_keys (sorted last) when the choice is dropped.
__device__ __forceinline__ int32_t load_key(const SortArgs& a, int32_t f) {
    int64_t at = f;
    if (a.ldi != a.k) {
        const int32_t t = f / a.k;
        at = t * a.ldi + (f - t * a.k);
    }
    const int64_t v =
        a.wide ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
    if (v >= 0 && v < a.n_keys) return static_cast<int32_t>(v);
    if (v >= 0) atomicOr(a.err, SPMM_DEVERR_INDEX);
    return a.n_keys;
}

// Input of a pass of more than a cluster: the ids, or the result of the launch
// before.
__device__ __forceinline__ int32_t pass_key(const SortArgs& a, int pass, int32_t i) {
    return pass ? ((pass & 1) ? a.keys0 : a.keys1)[i] : load_key(a, i);
}

__device__ __forceinline__ int32_t warp_scan(int32_t v, int lane) {  // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

struct SortShared {
    int32_t hist[kSortWarps][kBins];
    int32_t first[kBins];
    int32_t sums[kSortWarps];
};

// Digit counts of elements [i0, i1) into s.first.
__device__ __forceinline__ void count_digits(const SortArgs& a, int pass, int32_t i0, int32_t i1, SortShared& s) {
    const int bins = 1 << a.bits, shift = pass * a.bits;
    s.first[threadIdx.x] = 0;
    __syncthreads();
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads)
        atomicAdd(&s.first[(pass_key(a, pass, static_cast<int32_t>(i)) >> shift) & (bins - 1)], 1);
    __syncthreads();
}

// This thread's digit: `all` elements of it in the input, `below` of them in
// earlier CTAs.  Leaves the first place of the CTA's elements in s.first.
__device__ __forceinline__ void first_places(const SortArgs& a, int32_t all, int32_t below, bool write_offsets,
                                             SortShared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t incl = warp_scan(all, lane);
    if (lane == 31) s.sums[warp] = incl;
    __syncthreads();
    int32_t start = incl - all;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w)
        if (w < warp) start += s.sums[w];
    s.first[threadIdx.x] = start + below;
    if (write_offsets && static_cast<int>(threadIdx.x) <= a.n_keys) a.offsets[threadIdx.x] = start;
    __syncthreads();
}

// The elements of a CTA's tile on their way from one pass to the next, for
// inputs of one cluster at most (so an index fits 16 bits).
struct Exchange {
    int32_t key[kTile];
    uint16_t idx[kTile];
};
static_assert(kMaxCluster * kTile <= 65536, "indexes of a cluster's elements fit 16 bits");

// A thread's elements of a tile: consecutive ones per warp.  Key -1 past the end.
struct Items {
    int32_t key[kItems], idx[kItems];
    __device__ __forceinline__ void load(const SortArgs& a, int pass, int64_t tile, int32_t i1) {
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int64_t i = tile + (threadIdx.x >> 5) * (32 * kItems) + j * 32 + (threadIdx.x & 31);
            const int32_t at = static_cast<int32_t>(i);
            key[j] = i < i1 ? pass_key(a, pass, at) : -1;
            idx[j] = i < i1 && pass ? ((pass & 1) ? a.idx0 : a.idx1)[at] : at;
        }
    }
    __device__ __forceinline__ void load(const Exchange& x, int32_t n) {  // n elements of the tile
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int i = (threadIdx.x >> 5) * (32 * kItems) + j * 32 + (threadIdx.x & 31);
            key[j] = i < n ? x.key[i] : -1;
            idx[j] = i < n ? x.idx[i] : 0;
        }
    }
};

// Ranks of this warp's items among its equal digits, and the digits' counts in
// its row of s.hist.
__device__ __forceinline__ void rank_items(const SortArgs& a, int shift, const Items& it, int32_t (&rank)[kItems],
                                           SortShared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << a.bits;
    const uint32_t before = (1u << lane) - 1u;
    for (int b = lane; b < bins; b += 32) s.hist[warp][b] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const bool live = it.key[j] >= 0;
        const int digit = (it.key[j] >> shift) & (bins - 1);
        uint32_t peers = __ballot_sync(0xffffffffu, live);  // lanes with the same digit
#pragma unroll
        for (int b = 0; b < kDigitBits; ++b) {
            if (b < a.bits) {
                const uint32_t set = __ballot_sync(0xffffffffu, (digit >> b) & 1);
                peers &= (digit >> b) & 1 ? set : ~set;
            }
        }
        rank[j] = __popc(peers & before);
        if (live) rank[j] += s.hist[warp][digit];
        __syncwarp();
        if (live && (peers & before) == 0) s.hist[warp][digit] += __popc(peers);
        __syncwarp();
    }
}

// This thread's digit: its counts in the warps' rows become the elements before
// each warp's; returns their sum.
__device__ __forceinline__ int32_t scan_warps(SortShared& s, int32_t start) {
    int32_t c[kSortWarps], run = start;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) c[w] = s.hist[w][threadIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        s.hist[w][threadIdx.x] = run;
        run += c[w];
    }
    return run - start;
}

// Sends items to the places of an intermediate pass, in the tile of CTA
// p / kTile of the cluster (CLUSTER) or in this CTA's.
template <bool CLUSTER>
__device__ __forceinline__ void send_items(const SortArgs& a, int shift, const Items& it, const int32_t (&rank)[kItems],
                                           Exchange& x, const SortShared& s) {
    const int warp = threadIdx.x >> 5, bins = 1 << a.bits;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        if (it.key[j] < 0) continue;
        const int digit = (it.key[j] >> shift) & (bins - 1);
        const int32_t p = s.hist[warp][digit] + rank[j] + s.first[digit], at = p % kTile;
        if (CLUSTER) {
            const uint32_t cta = p / kTile;
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ptx::map_shared(ptx::smem_u32(&x.key[at]), cta)),
                         "r"(it.key[j])
                         : "memory");
            asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(ptx::map_shared(ptx::smem_u32(&x.idx[at]), cta)),
                         "h"(static_cast<uint16_t>(it.idx[j]))
                         : "memory");
        } else {
            x.key[at] = it.key[j];
            x.idx[at] = static_cast<uint16_t>(it.idx[j]);
        }
    }
}

// Writes a tile's items at first(digit) + hist + rank.
__device__ __forceinline__ void write_items(const SortArgs& a, int pass, const Items& it, const int32_t (&rank)[kItems],
                                            int32_t* next_table, const SortShared& s, bool add_first) {
    const int warp = threadIdx.x >> 5, bins = 1 << a.bits, shift = pass * a.bits;
    const bool last = pass + 1 == a.passes;
    const int tiles = a.chunk / kTile;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int32_t key = it.key[j], f = it.idx[j];
        if (key < 0) continue;
        const int digit = (key >> shift) & (bins - 1);
        const int32_t p = s.hist[warp][digit] + rank[j] + (add_first ? s.first[digit] : 0);
        if (last) {
            a.order[p] = f;
            a.pos[f] = key < a.n_keys ? p : -1;
        } else {
            ((pass & 1) ? a.idx1 : a.idx0)[p] = f;
        }
        int32_t* keys = last ? a.keys : (pass & 1) ? a.keys1 : a.keys0;
        if (keys) keys[p] = key;
        if (next_table) {
            const int32_t tile = p / kTile, cta = tiles == 1 ? tile : tile / tiles;
            atomicAdd(next_table + cta * bins + ((key >> (shift + a.bits)) & (bins - 1)), 1);
        }
    }
}

// Writes elements [i0, i1) at their places, a tile at a time; `it` holds the
// first tile and s.first the places of the first elements.
__device__ __forceinline__ void place_elements(const SortArgs& a, int pass, int32_t i0, int32_t i1, Items& it,
                                               int32_t* next_table, SortShared& s) {
    const int bins = 1 << a.bits;
    for (int64_t tile = i0; tile < i1; tile += kTile) {
        int32_t rank[kItems];
        rank_items(a, pass * a.bits, it, rank, s);
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < bins) {
            const int32_t start = s.first[threadIdx.x];
            s.first[threadIdx.x] = start + scan_warps(s, start);
        }
        __syncthreads();
        write_items(a, pass, it, rank, next_table, s, false);
        if (tile + kTile < i1) it.load(a, pass, tile + kTile, i1);
        __syncthreads();
    }
}

// All passes over one tile in one CTA; the digits' counts come with the ranks.
__global__ void __launch_bounds__(kSortThreads) route_small_kernel(const SortArgs a) {
    __shared__ SortShared s;
    __shared__ Exchange x;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    for (int pass = 0; pass < a.passes; ++pass) {
        Items it;
        int32_t rank[kItems];
        if (pass == 0)
            it.load(a, 0, 0, a.n);
        else
            it.load(x, a.n);
        rank_items(a, pass * a.bits, it, rank, s);
        __syncthreads();
        const int32_t all = static_cast<int>(threadIdx.x) < (1 << a.bits) ? scan_warps(s, 0) : 0;
        first_places(a, all, 0, a.passes == 1, s);
        if (pass + 1 < a.passes)
            send_items<false>(a, pass * a.bits, it, rank, x, s);
        else
            write_items(a, pass, it, rank, nullptr, s, true);
        __syncthreads();
    }
}

__device__ __forceinline__ int32_t ld_cluster(const int32_t* p, uint32_t rank) {
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ptx::map_shared(ptx::smem_u32(p), rank)) : "memory");
    return v;
}

// All passes over up to kMaxCluster tiles in one cluster, a tile per CTA.
__global__ void __launch_bounds__(kSortThreads) route_cluster_kernel(const SortArgs a) {
    __shared__ SortShared s;
    __shared__ Exchange x;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int cta = blockIdx.x, ctas = gridDim.x;  // the grid is one cluster
    const int32_t i0 = cta * kTile, i1 = min(a.n, i0 + kTile);
    for (int pass = 0; pass < a.passes; ++pass) {
        Items it;
        int32_t rank[kItems];
        if (pass == 0)
            it.load(a, 0, i0, i1);
        else
            it.load(x, i1 - i0);
        rank_items(a, pass * a.bits, it, rank, s);
        __syncthreads();
        const bool used = static_cast<int>(threadIdx.x) < (1 << a.bits);
        s.first[threadIdx.x] = used ? scan_warps(s, 0) : 0;
        ptx::cluster_sync_all();
        int32_t all = 0, below = 0;
        if (used) {
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) {
                const int32_t v = c < ctas ? ld_cluster(&s.first[threadIdx.x], c) : 0;
                all += v;
                if (c < cta) below += v;
            }
        }
        ptx::cluster_sync_all();  // every CTA has read the counts
        first_places(a, all, below, a.passes == 1 && cta == 0, s);
        if (pass + 1 == a.passes) {
            write_items(a, pass, it, rank, nullptr, s, true);
            break;
        }
        send_items<true>(a, pass * a.bits, it, rank, x, s);
        ptx::cluster_sync_all();  // this pass's results are written
    }
}

// Counts of the first pass, and zeros for those of the others.
__global__ void __launch_bounds__(kSortThreads) route_count_kernel(const SortArgs a) {
    __shared__ SortShared s;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int bins = 1 << a.bits;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    count_digits(a, 0, static_cast<int32_t>(i0), static_cast<int32_t>(min(i0 + a.chunk, int64_t(a.n))), s);
    if (static_cast<int>(threadIdx.x) < bins) {
        int32_t* mine = a.table + blockIdx.x * bins + threadIdx.x;
        *mine = s.first[threadIdx.x];
        for (int pass = 1; pass < a.passes; ++pass) mine[pass * gridDim.x * bins] = 0;
    }
}

__global__ void __launch_bounds__(kSortThreads) route_place_kernel(const SortArgs a, int pass) {
    __shared__ SortShared s;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int bins = 1 << a.bits, cta = blockIdx.x, ctas = gridDim.x;
    int32_t* table = a.table + pass * ctas * bins;
    const int32_t i0 = cta * a.chunk, i1 = static_cast<int32_t>(min(int64_t(i0) + a.chunk, int64_t(a.n)));
    Items it;  // in flight while the counts are added up
    it.load(a, pass, i0, i1);
    int32_t all = 0, below = 0;
    // digits that occur: the last pass has no key above n_keys
    const int used = pass + 1 == a.passes ? (a.n_keys >> (pass * a.bits)) + 1 : bins;
    if (static_cast<int>(threadIdx.x) < used) {
        // 16 loads in flight; every CTA starts at its own row, or they would all queue at one L2 slice
        for (int c0 = 0; c0 < ctas; c0 += 16) {
            int32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int c = c0 + i + cta < ctas ? c0 + i + cta : c0 + i + cta - ctas;
                v[i] = c0 + i < ctas ? table[c * bins + threadIdx.x] : 0;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                all += v[i];
                if (c0 + i + cta >= ctas) below += v[i];  // row c0 + i + cta - ctas, before cta's
            }
        }
    }
    first_places(a, all, below, a.passes == 1 && cta == 0, s);
    place_elements(a, pass, i0, i1, it,
                   pass + 1 < a.passes ? table + ctas * bins : nullptr, s);
}

// More than one pass: offsets[e] is the number of sorted keys below e.  A CTA
// finds the place of its first key 256 probes at a time; its threads search on
// from there in doubling steps, on lines that are then in L1.  (Counting with
// atomics and scanning n_keys counts in the sort's few CTAs took 45 us for
// 131072 keys.)
constexpr int kOffsetThreads = 256;

__global__ void __launch_bounds__(kOffsetThreads)
    route_offsets_kernel(const int32_t* sorted, int32_t n, int32_t n_keys, int32_t* offsets) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t e0 = static_cast<int64_t>(blockIdx.x) * kOffsetThreads, e = e0 + threadIdx.x;
    int64_t lo = 0, hi = n;  // the answer for e0 lies in [lo, hi]
    while (lo < hi) {
        const int64_t step = (hi - lo + kOffsetThreads - 1) / kOffsetThreads, at = lo + threadIdx.x * step;
        const int64_t below = __syncthreads_count(at < hi && sorted[at] < e0);
        hi = min(hi, lo + below * step);
        if (below) lo += (below - 1) * step + 1;
    }
    if (e > n_keys) return;
    int64_t step = 1;
    while (lo + step <= n && sorted[lo + step - 1] < e) {
        lo += step;
        step *= 2;
    }
    hi = min(int64_t(n), lo + step - 1);
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (sorted[mid] < e)
            lo = mid + 1;
        else
            hi = mid;
    }
    offsets[e] = static_cast<int32_t>(lo);
}

// ---------------------------------------------------------------- rows
constexpr int kRowThreads = 128;       // products and gradient (256: 332 us where 128 take 324, 16384 x 4 x 3584 fp16)
constexpr int kDispatchThreads = 512;  // copies (256: 179 us, 512: 177 us, 16384 x 8 x 4096 bf16)
constexpr int kBatch = 4;  // rows of a token in flight per thread

struct RowArgs {
    const int32_t *pos, *offsets;
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
    for (int64_t p = a.offsets[a.n_keys] + static_cast<int64_t>(blockIdx.x); p < a.T * a.k; p += gridDim.x)
        for (int64_t c = threadIdx.x * V; c < a.H; c += blockDim.x * V)
            Vec<T, V>::store_cs(out + p * a.ldo + c, Vec<T, V>::zero());
}

// One CTA per token: its row is read once and written at its k places.
template <typename T, int V>
__global__ void __launch_bounds__(kDispatchThreads) dispatch_kernel(const RowArgs a) {
    using X = Cols<T, V, 2>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const T* x = static_cast<const T*>(a.a) + blockIdx.x * a.lda;
    T* out = static_cast<T*>(a.out);
    const int32_t* pos = a.pos + static_cast<int64_t>(blockIdx.x) * a.k;
    const int step = blockDim.x * V;
    for (int64_t c = threadIdx.x * V; c < a.H; c += X::U * step) {
        typename X::Raw r[X::U];
        X::load(r, x, c, a.H, step);
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = pos[j];
            if (p >= 0) X::store_cs(out + p * a.ldo, r, c, a.H, step);
        }
    }
    zero_tail<T, V>(a, out);
}

// One CTA per token: its k rows summed in fp32 with their weights, j ascending,
// and rounded once.  Four rows are in flight per thread.
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const RowArgs a) {
    using X = Cols<T, V>;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const T* ys = static_cast<const T*>(a.a);
    T* y = static_cast<T*>(a.out) + blockIdx.x * a.ldo;
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * a.k;
    const int step = blockDim.x * V;
    int64_t p[kBatch];  // places of the batch's rows, and their weights
    float w[kBatch];
    const auto choices = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            p[j] = j0 + j < a.k ? a.pos[f0 + j0 + j] : -1;
            w[j] = a.w && p[j] >= 0 ? a.w[f0 + j0 + j] : 1.f;
        }
    };
    // up to four choices are read once where the moves are narrow and the columns take
    // many rounds (4095: 76 us, read every round 81); at full width the registers
    // cost more than the reads (4096: 53 us, read every round 51)
    constexpr bool kOnce = X::U > 1;
    if (kOnce) choices(0);
    for (int64_t c = threadIdx.x * V; c < a.H; c += X::U * step) {
        float acc[X::N] = {};
        for (int j0 = 0; j0 < a.k; j0 += kBatch) {
            if (!kOnce || a.k > kBatch) choices(j0);
            typename X::Raw r[kBatch][X::U];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (p[j] >= 0)
                    X::load(r[j], ys + p[j] * a.lda, c, a.H, step);
                else
                    X::clear(r[j]);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (p[j] < 0) continue;  // not 0 * w: a weight may be infinite
                float v[X::N];
                X::unpack(r[j], v);
#pragma unroll
                for (int i = 0; i < X::N; ++i) acc[i] = fmaf(w[j], v[i], acc[i]);
            }
        }
        typename X::Raw o[X::U];
        X::pack(o, acc);
        X::store(y, o, c, a.H, step);
    }
}

// One CTA per token: dys = w dy at its k places and the k dot products of dy
// with ys, each summed in fp32 per thread, then over the CTA in a fixed order.
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const RowArgs a) {
    using X = Cols<T, V>;
    __shared__ float part[kBatch][kRowThreads / 32];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const T* dy = static_cast<const T*>(a.a) + blockIdx.x * a.lda;
    const T* ys = static_cast<const T*>(a.b);
    T* dys = static_cast<T*>(a.out);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * a.k;
    const int step = blockDim.x * V;
    for (int j0 = 0; j0 < a.k; j0 += kBatch) {
        int64_t p[kBatch];
        float w[kBatch], dot[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            p[j] = j0 + j < a.k ? a.pos[f0 + j0 + j] : -1;
            w[j] = p[j] >= 0 ? a.w[f0 + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int64_t c = threadIdx.x * V; c < a.H; c += X::U * step) {
            typename X::Raw r[kBatch][X::U], q[X::U];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (p[j] >= 0)
                    X::load(r[j], ys + p[j] * a.ldb, c, a.H, step);
                else
                    X::clear(r[j]);
            }
            X::load(q, dy, c, a.H, step);
            float d[X::N];
            X::unpack(q, d);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (p[j] < 0) continue;
                float v[X::N];
                X::unpack(r[j], v);
#pragma unroll
                for (int i = 0; i < X::N; ++i) {
                    dot[j] = fmaf(d[i], v[i], dot[j]);
                    v[i] = w[j] * d[i];
                }
                typename X::Raw o[X::U];
                X::pack(o, v);
                X::store_cs(dys + p[j] * a.ldo, o, c, a.H, step);
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
#pragma unroll
            for (int s = 16; s; s >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
            if (lane == 0) part[j][warp] = dot[j];
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < kBatch && j0 + static_cast<int>(threadIdx.x) < a.k) {
            float s = 0.f;
            for (int i = 0; i < warps; ++i) s += part[threadIdx.x][i];
            a.dw[f0 + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
    zero_tail<T, V>(a, dys);
}

}  // namespace

namespace {
struct SortPlan {
    int passes, bits, ctas, chunk;
};
SortPlan sort_plan(int64_t n, int64_t n_keys) {
    SortPlan p{};
    int total = 1;  // bits of the largest key, n_keys itself
    while (n_keys >> total) ++total;
    p.passes = (total + kDigitBits - 1) / kDigitBits;
    p.bits = (total + p.passes - 1) / p.passes;
    const int64_t tiles = n ? (n + kTile - 1) / kTile : 1;
    const int64_t per = (tiles + kMaxCtas - 1) / kMaxCtas;
    p.chunk = static_cast<int>(per * kTile);
    p.ctas = static_cast<int>((tiles + per - 1) / per);
    return p;
}
}  // namespace

size_t route_workspace_bytes(int64_t T, int32_t k, int64_t n_keys) {
    const int64_t n = T * k;
    const SortPlan p = sort_plan(n, n_keys);
    return (p.passes > 1 ? static_cast<size_t>(n) * 16 : 0) +
           (p.ctas > kMaxCluster ? static_cast<size_t>(p.ctas) * sizeof(int32_t) * p.passes << p.bits : 0);
}

spmm_status launch_build_route(const void* ids, int32_t id_bytes, int64_t ldi, const spmm_route_t* R, void* ws,
                               cudaStream_t s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return SPMM_ERR_CUDA;
    const int32_t n = static_cast<int32_t>(R->T * R->k);
    const SortPlan p = sort_plan(n, R->n_keys);
    SortArgs a{};
    a.ids = ids;
    a.ldi = ldi;
    a.wide = id_bytes == 8;
    a.k = R->k;
    a.n = n;
    a.n_keys = static_cast<int32_t>(R->n_keys);
    a.passes = p.passes;
    a.bits = p.bits;
    a.chunk = p.chunk;
    a.order = R->order;
    a.pos = R->pos;
    a.offsets = R->offsets;
    a.keys = R->keys;
    int32_t* w = static_cast<int32_t*>(ws);
    if (p.passes > 1) {
        a.keys0 = w;
        a.idx0 = w + static_cast<int64_t>(n);
        a.keys1 = w + 2 * static_cast<int64_t>(n);
        a.idx1 = w + 3 * static_cast<int64_t>(n);
        if (!a.keys) a.keys = (p.passes & 1) ? a.keys0 : a.keys1;  // the offsets are searched in them
        w += 4 * static_cast<int64_t>(n);
    }
    a.table = w;
    a.err = dev->err;
    trace_begin(SPMM_KERNEL_ROUTE, s);
    cudaError_t e = cudaSuccess;
    if (p.ctas == 1) {
        e = launch_chained(route_small_kernel, 1, kSortThreads, 0, 1, s, a);
    } else if (p.ctas <= kMaxCluster) {
        e = launch_chained(route_cluster_kernel, p.ctas, kSortThreads, 0, p.ctas, s, a);
    } else {
        e = launch_chained(route_count_kernel, p.ctas, kSortThreads, 0, 1, s, a);
        for (int pass = 0; pass < p.passes && e == cudaSuccess; ++pass)
            e = launch_chained(route_place_kernel, p.ctas, kSortThreads, 0, 1, s, a, pass);
    }
    if (p.passes > 1 && e == cudaSuccess)
        e = launch_chained(route_offsets_kernel, static_cast<unsigned>(R->n_keys / kOffsetThreads + 1),
                           kOffsetThreads, 0, 1, s,
                           a.keys, n, a.n_keys, a.offsets);
    trace_end(SPMM_KERNEL_ROUTE, s);
    return cuda_status(e);
}

static RowArgs row_args(const spmm_route_t* R, int64_t H) {
    RowArgs a{};
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
    const Operand o[] = {{x, ldx, es}, {xs, ldxs, es}};
    const int v = row_width(o, H);
    const unsigned grid = static_cast<unsigned>(R->T);
    const int threads = row_threads(H, 16 / es, kDispatchThreads);
    trace_begin(SPMM_KERNEL_ROWS, s);
    cudaError_t e;
    SPMM_ROWS_TYPED(e, dtype, v, dispatch_kernel, grid, threads, s, a);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(e);
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
    const Operand o[] = {{ys, ldys, es}, {y, ldy, es}};
    const int v = row_width(o, H);
    const unsigned grid = static_cast<unsigned>(R->T);
    const int threads = row_threads(H, 16 / es, kRowThreads);
    trace_begin(SPMM_KERNEL_ROWS, s);
    cudaError_t e;
    SPMM_ROWS_TYPED(e, dtype, v, combine_kernel, grid, threads, s, a);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(e);
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
    const Operand o[] = {{dy, lddy, es}, {ys, ldys, es}, {dys, lddys, es}};
    const int v = row_width(o, H);
    const unsigned grid = static_cast<unsigned>(R->T);
    const int threads = row_threads(H, 16 / es, kRowThreads);
    trace_begin(SPMM_KERNEL_ROWS, s);
    cudaError_t e;
    SPMM_ROWS_TYPED(e, dtype, v, combine_grad_kernel, grid, threads, s, a);
    trace_end(SPMM_KERNEL_ROWS, s);
    return cuda_status(e);
}

}  // namespace spmm
