// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out_i  = scale W[id_i]                          (padding: a row of zeros)
//   gW_v   = scale sum over {i : id_i = v} of g_i   (a row of zeros if none)
//
// Both are bound by HBM: the lookup moves the distinct rows of W in and n d
// elements out, the gradient n d elements in and V d out.
//
// The gradient must not depend on the order in which threads run, so it uses no
// floating-point atomics: the (id, position) pairs are put in order by a stable
// radix sort, and the sums follow the sorted order in fixed groups.
//
// Measured: the lookup of 262144 fp32 rows of 512 takes 101 us (6.1 TB/s of the
// distinct rows and the output).  The gradient of 262144 bf16 rows of 1024 with ids
// as frequent as words, V = 65536, takes 166 us: sorting 40 us, beside which gW is
// cleared, sums 107 us (5.6 TB/s), joining 17 us (a chain of dependent reads).
#include <initializer_list>

#include <cooperative_groups.h>

#include "../../include/nrnn.h"
#include "nrnn_device.cuh"
#include "nrnn_internal.h"
#include "rows.cuh"

namespace cg = cooperative_groups;

namespace nrnn {
namespace {

// A warp works on 32 VEC consecutive columns (a slab) of a row.
constexpr int GROUP_ROWS = 4;      // rows of one warp of the lookup
constexpr int EMBED_THREADS = 128;

template <typename Id> __device__ __forceinline__ int64_t id_at(const void *ids, int64_t i) {
    return static_cast<int64_t>(static_cast<const Id *>(ids)[i]);
}

// ------------------------------------------------------------------ the lookup
// A warp copies one slab of GROUP_ROWS rows, all loads before the first store: with
// one row a warp the loads in flight would not cover the memory's latency.
// An id outside [0, V) that is not the padding id gives a row of NaN.
template <typename T, int VEC, typename Id>
__global__ void __launch_bounds__(EMBED_THREADS)
    k_embedding(const void *__restrict__ ids, const T *__restrict__ W, T *__restrict__ out,
                int64_t n, int64_t V, int64_t d, int slabs, int64_t pad, float scale) {
    wait_for_prerequisites();
    const int lane = threadIdx.x & 31;
    const int64_t item =
        blockIdx.x * static_cast<int64_t>(EMBED_THREADS / 32) + (threadIdx.x >> 5);
    const int64_t r0 = item / slabs * GROUP_ROWS;
    if (r0 >= n) return;
    const int64_t c = static_cast<int64_t>(item % slabs) * (32 * VEC) + lane * VEC;
    const int rows = n - r0 < GROUP_ROWS ? static_cast<int>(n - r0) : GROUP_ROWS;
    int64_t id = -1;
    if (lane < rows) id = id_at<Id>(ids, r0 + lane);
    int64_t ks[GROUP_ROWS];
#pragma unroll
    for (int r = 0; r < GROUP_ROWS; ++r) ks[r] = __shfl_sync(FULL_MASK, id, r);
    if (c >= d) return;
    float v[GROUP_ROWS][VEC];
#pragma unroll
    for (int r = 0; r < GROUP_ROWS; ++r) {
        const int64_t k = ks[r];
        const bool padding = pad >= 0 && k == pad;
        const float fill = padding ? 0.f : __int_as_float(0x7fffffff);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[r][e] = fill;
        if (r < rows && !padding && k >= 0 && k < V) load_f32<T, VEC>(W + k * d + c, v[r]);
    }
#pragma unroll
    for (int r = 0; r < GROUP_ROWS; ++r) {
        if (r >= rows) break;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[r][e] *= scale;
        store_f32<T, VEC>(out + (r0 + r) * d + c, v[r]);
    }
}

// -------------------------------------------------------------------- the sort
// Stable least-significant-digit radix sort of (id, position), up to 9 bits a
// pass.  Each pass is two launches over at most SORT_CTAS contiguous parts of the
// input: k_sort_count leaves the parts' digit counts, and k_sort_place adds up
// the counts before its own part (all parts' for lower digits, earlier parts'
// for equal ones), ranks its pairs and writes them.  Ranks follow (part, round,
// warp, step, lane) = input order.  A tile's pairs are put in order in shared memory first, so that a
// digit's run leaves as whole lines.  (All passes in one cluster of 16 CTAs took
// 56 us for 262144 ids, bound by those SMs; up to 32768 ids it is faster.)
// Ids that take no part (padding, out of range) get the key V and sort last.
//
// The launches' further CTAs clear gW meanwhile, a share each.
constexpr int SORT_CTAS = 152;
constexpr int SORT_THREADS = 512, SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_MAX_BITS = 9, SORT_DIGITS = 1 << SORT_MAX_BITS;
constexpr int SORT_STEPS = 4;                              // pairs of a thread in a tile
constexpr int SORT_TILE = SORT_STEPS * SORT_THREADS;
constexpr int CLEAR_CTAS = 304;

struct SortArgs {
    const void *ids;
    uint32_t n, V;
    int64_t pad;
    const uint32_t *kin, *pin;   // the pass's pairs; null: the ids themselves
    uint32_t *kout, *pout;
    uint32_t *count;             // [ctas][SORT_DIGITS]
    uint32_t *spanning;          // the list of long segments: count, then {chunk, id}
    int ctas, rounds;            // parts, and tiles of a part
    int shift, bits;
    uint4 *clear;                // this launch's share of gW
    int64_t clear16;
    unsigned char *ends[2];      // the bytes of gW before and after its 16-byte pieces
    int end_bytes[2];
};

struct SortShared {
    uint32_t cnt[SORT_WARPS][SORT_DIGITS];
    uint32_t start[SORT_DIGITS];     // first place of a digit in the tile
    uint32_t base[SORT_DIGITS];      // and in the output
    uint32_t sums[2][4][SORT_DIGITS];
    uint32_t key[SORT_TILE], pos[SORT_TILE];
    uint32_t warp_sum[SORT_WARPS];
};

// lanes that hold the same digit (out-of-range lanes share one above the digits):
// one ballot per bit, independent of one another, which is faster than match.any
// on digits that mostly differ
__device__ __forceinline__ unsigned same_digit(uint32_t digit) {
    unsigned peers = FULL_MASK;
#pragma unroll
    for (int i = 0; i <= SORT_MAX_BITS; ++i) {
        const bool one = (digit >> i) & 1u;
        const unsigned vote = __ballot_sync(FULL_MASK, one);
        peers &= one ? vote : ~vote;
    }
    return peers;
}

template <typename Id>
__device__ __forceinline__ void sort_load(const SortArgs &a, uint64_t i0, uint32_t (&k)[SORT_STEPS]) {
#pragma unroll
    for (int j = 0; j < SORT_STEPS; ++j) {
        const uint64_t i = i0 + j * 32;
        k[j] = a.V;
        if (i >= a.n) continue;
        if (a.kin != nullptr) {
            k[j] = a.kin[i];
        } else {
            const int64_t id = id_at<Id>(a.ids, i);
            if (id >= 0 && id < a.V && id != a.pad) k[j] = static_cast<uint32_t>(id);
        }
    }
}

// counts the warp's digits; rank: a pair's rank among its warp's equal digits
__device__ __forceinline__ void sort_rank(uint32_t *mine, const uint32_t (&k)[SORT_STEPS], uint64_t i0,
                                          uint64_t n, int shift, uint32_t mask,
                                          uint32_t (&rank)[SORT_STEPS]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < SORT_STEPS; ++j) {
        const bool in = i0 + j * 32 < n;
        const uint32_t digit = in ? (k[j] >> shift) & mask : SORT_DIGITS;
        const unsigned peers = same_digit(digit);
        const uint32_t before = in ? mine[digit] : 0;
        __syncwarp();
        rank[j] = before + __popc(peers & ((1u << lane) - 1u));
        if (in && lane == __ffs(peers) - 1) mine[digit] = before + __popc(peers);
        __syncwarp();
    }
}

__device__ __forceinline__ void sort_zero(SortShared &s) {
    uint4 *p = reinterpret_cast<uint4 *>(s.cnt);
#pragma unroll
    for (int i = 0; i < SORT_WARPS * SORT_DIGITS / 4 / SORT_THREADS; ++i)
        p[i * SORT_THREADS + threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
}

// the warps' counts of this thread's digit become counts before each warp; returns their sum
__device__ __forceinline__ uint32_t sort_scan_warps(SortShared &s) {
    uint32_t c[SORT_WARPS], run = 0;
#pragma unroll
    for (int v = 0; v < SORT_WARPS; ++v) c[v] = s.cnt[v][threadIdx.x];
#pragma unroll
    for (int v = 0; v < SORT_WARPS; ++v) {
        s.cnt[v][threadIdx.x] = run;
        run += c[v];
    }
    return run;
}

// exclusive scan of v over the digits (one per thread)
__device__ __forceinline__ uint32_t sort_scan_digits(SortShared &s, uint32_t v) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(FULL_MASK, incl, o);
        if (lane >= o) incl += t;
    }
    __syncthreads();   // warp_sum is free
    if (lane == 31) s.warp_sum[w] = incl;
    __syncthreads();
    uint32_t lower = 0;
#pragma unroll
    for (int v2 = 0; v2 < SORT_WARPS; ++v2) lower += v2 < w ? s.warp_sum[v2] : 0;
    return lower + incl - v;
}
static_assert(SORT_THREADS == SORT_DIGITS, "one digit per thread");
static_assert(CLEAR_CTAS % 16 == 0, "whole clusters of the clearing CTAs");

__device__ __forceinline__ void clear_share(const SortArgs &a, int cta) {
    const int64_t step = static_cast<int64_t>(CLEAR_CTAS) * SORT_THREADS;
    for (int64_t i = static_cast<int64_t>(cta) * SORT_THREADS + threadIdx.x; i < a.clear16; i += step)
        a.clear[i] = make_uint4(0u, 0u, 0u, 0u);
    if (cta == 0)
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (static_cast<int>(threadIdx.x) < a.end_bytes[q]) a.ends[q][threadIdx.x] = 0;
}

template <typename Id>
__global__ void __launch_bounds__(SORT_THREADS) k_sort_count(const SortArgs a) {
    extern __shared__ __align__(16) unsigned char sort_smem[];
    SortShared &s = *reinterpret_cast<SortShared *>(sort_smem);
    dependents_may_launch();
    wait_for_prerequisites();
    if (static_cast<int>(blockIdx.x) >= a.ctas) return clear_share(a, blockIdx.x - a.ctas);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t k[SORT_STEPS], rank[SORT_STEPS];
    const uint64_t part = static_cast<uint64_t>(blockIdx.x) * a.rounds * SORT_TILE;
    sort_zero(s);
    __syncthreads();
    for (int r = 0; r < a.rounds; ++r) {
        const uint64_t i0 = part + r * static_cast<uint64_t>(SORT_TILE) + w * (32 * SORT_STEPS) + lane;
        sort_load<Id>(a, i0, k);
        sort_rank(s.cnt[w], k, i0, a.n, a.shift, (1u << a.bits) - 1u, rank);
    }
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (int v = 0; v < SORT_WARPS; ++v) all += s.cnt[v][threadIdx.x];
    a.count[blockIdx.x * SORT_DIGITS + threadIdx.x] = all;
}

// ranks a tile's pairs and writes them from s.base on
__device__ __forceinline__ void sort_place(SortShared &s, const SortArgs &a, uint64_t tile,
                                           uint64_t i0, const uint32_t (&k)[SORT_STEPS]) {
    const int w = threadIdx.x >> 5;
    const uint32_t mask = (1u << a.bits) - 1u;
    uint32_t p[SORT_STEPS], rank[SORT_STEPS];
#pragma unroll
    for (int j = 0; j < SORT_STEPS; ++j) {
        const uint64_t i = i0 + j * 32;
        p[j] = a.kin != nullptr && i < a.n ? a.pin[i] : static_cast<uint32_t>(i);
    }
    sort_rank(s.cnt[w], k, i0, a.n, a.shift, mask, rank);
    __syncthreads();
    const uint32_t own = sort_scan_warps(s);
    const uint32_t start = sort_scan_digits(s, own);
    s.start[threadIdx.x] = start;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < SORT_STEPS; ++j) {
        if (i0 + j * 32 >= a.n) continue;
        const uint32_t digit = (k[j] >> a.shift) & mask;
        const uint32_t at = s.start[digit] + s.cnt[w][digit] + rank[j];
        s.key[at] = k[j];
        s.pos[at] = p[j];
    }
    __syncthreads();
    const uint32_t have = tile >= a.n ? 0 : a.n - tile < SORT_TILE ? static_cast<uint32_t>(a.n - tile) : SORT_TILE;
#pragma unroll
    for (int j = 0; j < SORT_STEPS; ++j) {
        const uint32_t i = j * SORT_THREADS + threadIdx.x;
        if (i >= have) continue;
        const uint32_t key = s.key[i], digit = (key >> a.shift) & mask;
        const uint32_t at = s.base[digit] + i - s.start[digit];
        a.kout[at] = key;
        a.pout[at] = s.pos[i];
    }
    __syncthreads();
    s.base[threadIdx.x] += own;   // the next tile's
}

template <typename Id>
__global__ void __launch_bounds__(SORT_THREADS) k_sort_place(const SortArgs a) {
    extern __shared__ __align__(16) unsigned char sort_smem[];
    SortShared &s = *reinterpret_cast<SortShared *>(sort_smem);
    dependents_may_launch();
    wait_for_prerequisites();
    if (static_cast<int>(blockIdx.x) >= a.ctas) return clear_share(a, blockIdx.x - a.ctas);
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    if (blockIdx.x == 0 && t == 0) *a.spanning = 0;
    // digit counts: 128 threads a part (four digits each), four parts at a time
    uint4 before = make_uint4(0u, 0u, 0u, 0u), all = before;
    const uint4 *count = reinterpret_cast<const uint4 *>(a.count) + (t & 127);
#pragma unroll 8
    for (int c = t >> 7; c < a.ctas; c += 4) {
        const uint4 v = count[c * (SORT_DIGITS / 4)];
        all.x += v.x; all.y += v.y; all.z += v.z; all.w += v.w;
        if (c < static_cast<int>(blockIdx.x)) {
            before.x += v.x; before.y += v.y; before.z += v.z; before.w += v.w;
        }
    }
    reinterpret_cast<uint4 *>(s.sums[0][t >> 7])[t & 127] = before;
    reinterpret_cast<uint4 *>(s.sums[1][t >> 7])[t & 127] = all;
    __syncthreads();
    uint32_t lower = 0, total = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        lower += s.sums[0][q][t];
        total += s.sums[1][q][t];
    }
    s.base[t] = sort_scan_digits(s, total) + lower;
    const uint64_t part = static_cast<uint64_t>(blockIdx.x) * a.rounds * SORT_TILE;
    for (int r = 0; r < a.rounds; ++r) {
        const uint64_t tile = part + r * static_cast<uint64_t>(SORT_TILE);
        const uint64_t i0 = tile + w * (32 * SORT_STEPS) + lane;
        uint32_t k[SORT_STEPS];
        sort_load<Id>(a, i0, k);
        sort_zero(s);
        __syncthreads();
        sort_place(s, a, tile, i0, k);
    }
}

// Up to SORT_CLUSTER tiles: one cluster with a tile per CTA does every pass in
// one launch.  A pass's counts and pairs are exchanged through distributed shared
// memory; only the sorted pairs go to global memory.  (30001 ids: two launches a
// pass took 23 us; here 15.)
constexpr int SORT_CLUSTER = 16;   // above the portable 8: allowed by attribute

struct ClusterSortShared {
    SortShared s;
    uint32_t key[2][SORT_TILE], pos[2][SORT_TILE];
    uint32_t total[SORT_DIGITS];
};

template <typename Id>
__global__ void __launch_bounds__(SORT_THREADS) k_sort_cluster(SortArgs a, int passes) {
    extern __shared__ __align__(16) unsigned char sort_smem[];
    ClusterSortShared &c = *reinterpret_cast<ClusterSortShared *>(sort_smem);
    SortShared &s = c.s;
    dependents_may_launch();
    wait_for_prerequisites();
    if (static_cast<int>(blockIdx.x) >= a.ctas) return clear_share(a, blockIdx.x - a.ctas);
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t r = cluster.block_rank();
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    const uint32_t mask = (1u << a.bits) - 1u;
    if (r == 0 && t == 0) *a.spanning = 0;
    const uint32_t slot = w * (32 * SORT_STEPS) + lane;          // + 32 j: this thread's pairs
    const uint64_t i0 = static_cast<uint64_t>(r) * SORT_TILE + slot;
    uint32_t k[SORT_STEPS], p[SORT_STEPS], rank[SORT_STEPS];
    sort_load<Id>(a, i0, k);
#pragma unroll
    for (int j = 0; j < SORT_STEPS; ++j) p[j] = static_cast<uint32_t>(i0) + j * 32;
    for (int q = 0; q < passes; ++q) {
        const int shift = q * a.bits;
        sort_zero(s);
        __syncthreads();
        sort_rank(s.cnt[w], k, i0, a.n, shift, mask, rank);
        __syncthreads();
        c.total[t] = sort_scan_warps(s);
        cluster.sync();
        uint32_t before = 0, all = 0;
        uint32_t theirs[SORT_CLUSTER];   // all remote reads in flight together
#pragma unroll
        for (int o = 0; o < SORT_CLUSTER; ++o)
            theirs[o] = o < a.ctas ? *cluster.map_shared_rank(c.total + t, o) : 0;
#pragma unroll
        for (int o = 0; o < SORT_CLUSTER; ++o) {
            before += o < static_cast<int>(r) ? theirs[o] : 0;
            all += theirs[o];
        }
        const uint32_t base = sort_scan_digits(s, all) + before;
        s.base[t] = base;
        __syncthreads();
        uint32_t *to_key = c.key[q & 1], *to_pos = c.pos[q & 1];
#pragma unroll
        for (int j = 0; j < SORT_STEPS; ++j) {
            if (i0 + j * 32 >= a.n) continue;
            const uint32_t digit = (k[j] >> shift) & mask;
            const uint32_t at = s.base[digit] + s.cnt[w][digit] + rank[j];
            *cluster.map_shared_rank(to_key + at % SORT_TILE, at / SORT_TILE) = k[j];
            *cluster.map_shared_rank(to_pos + at % SORT_TILE, at / SORT_TILE) = p[j];
        }
        cluster.sync();   // the pairs have arrived; `total` is free again
#pragma unroll
        for (int j = 0; j < SORT_STEPS; ++j) {
            k[j] = to_key[slot + j * 32];
            p[j] = to_pos[slot + j * 32];
        }
    }
#pragma unroll
    for (int j = 0; j < SORT_STEPS; ++j) {
        if (i0 + j * 32 >= a.n) continue;
        a.kout[i0 + j * 32] = k[j];
        a.pout[i0 + j * 32] = p[j];
    }
}

template <typename Id>
cudaError_t sort_ids(SortArgs a, uint32_t *const (&key)[2], uint32_t *const (&pos)[2], int passes,
                     unsigned char *clear, int64_t clear16, bool clears, cudaStream_t stream) {
    static std::atomic<unsigned long long> configured{0};
    constexpr int smem = sizeof(SortShared);
    cudaError_t e = once_per_device(configured, [](int) {
        cudaError_t r = cudaFuncSetAttribute(k_sort_count<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(k_sort_place<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(k_sort_cluster<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     sizeof(ClusterSortShared));
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(k_sort_cluster<Id>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
    });
    if (e != cudaSuccess) return e;
    const int more = clears ? CLEAR_CTAS : 0;
    const int64_t tiles = (static_cast<int64_t>(a.n) + SORT_TILE - 1) / SORT_TILE;
    if (tiles <= SORT_CLUSTER) {
        a.ctas = 1;
        while (a.ctas < tiles) a.ctas *= 2;   // divides the clearing CTAs
        a.kout = key[1];
        a.pout = pos[1];
        a.clear = reinterpret_cast<uint4 *>(clear);
        a.clear16 = clear16;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(a.ctas + more));
        cfg.blockDim = dim3(SORT_THREADS);
        cfg.dynamicSmemBytes = sizeof(ClusterSortShared);
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(a.ctas);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, k_sort_cluster<Id>, a, passes);
    }
    a.rounds = static_cast<int>((tiles + SORT_CTAS - 1) / SORT_CTAS);
    a.ctas = static_cast<int>((tiles + a.rounds - 1) / a.rounds);
    const int64_t share = (clear16 + 2 * passes - 1) / (2 * passes);
    int64_t cleared = 0;
    for (int q = 0; q < passes; ++q) {
        a.shift = q * a.bits;
        const int to = (passes - 1 - q) & 1 ? 0 : 1;   // the last pass writes [1]
        a.kin = q == 0 ? nullptr : key[to ^ 1];
        a.pin = pos[to ^ 1];
        a.kout = key[to];
        a.pout = pos[to];
        for (int half = 0; half < 2; ++half) {
            a.clear = reinterpret_cast<uint4 *>(clear) + cleared;
            a.clear16 = clear16 - cleared < share ? clear16 - cleared : share;
            cleared += a.clear16;
            e = launch_dependent(half == 0 ? k_sort_count<Id> : k_sort_place<Id>,
                                 a.ctas + more, SORT_THREADS, smem, stream, a);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

// ---------------------------------------------------------------- the gradient
// A warp sums one slab of a chunk of consecutive sorted pairs.  It writes the
// segments (the pairs of one id) that begin in its chunk, going on into the next
// chunk for one that crosses the edge.  Only a long segment, one that fills at
// least one whole chunk, is cut at the chunks' edges: each chunk leaves its part
// of the sum in fp32 (slot 0: the segment came in from the left, slot 1: it
// begins here), and k_embed_join adds the parts in order.  With ids as frequent
// as words, only some hundred ids are that long.  Chunks have 32 pairs, or (where
// those are more than the SMs hold warps for) up to MAX_CHUNK, which leaves fewer
// parts: at 262144 pairs of 1024 columns joining took 46 us at 32.
constexpr int MIN_CHUNK = 32, MAX_CHUNK = 64;
constexpr int64_t FEW_WARPS = 10000;

template <typename T, int VEC>
__device__ __forceinline__ void write_row(T *p, float (&acc)[VEC], float scale, bool accumulate) {
    float o[VEC];
    if (accumulate) {
        load_f32<T, VEC>(p, o);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = fmaf(acc[e], scale, o[e]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = acc[e] * scale;
    }
    store_f32<T, VEC>(p, o);
}

// Rows on their way: each lane copies its own VEC columns to its own place in
// shared memory (cp.async) and reads them back itself, so a warp keeps 16 rows
// in flight in no registers and needs no barrier.  (Eight rows in registers: 126
// registers, 16 warps an SM, 2.8 TB/s on 262144 x 1024 bf16.)
constexpr int BATCH = 8;             // rows of one commit group
constexpr int RING = 2 * BATCH;

template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src),
                     "n"(BYTES >= 4 ? BYTES : 4)
                     : "memory");
}

template <typename T, int VEC>
__global__ void __launch_bounds__(EMBED_THREADS)
    k_embed_grad(const uint32_t *__restrict__ key, const uint32_t *__restrict__ pos,
                 const T *__restrict__ g, T *__restrict__ gW, float *__restrict__ part,
                 uint32_t *__restrict__ spanning, uint32_t n, uint32_t V, int64_t d, int L, int slabs,
                 int64_t items, float scale, bool accumulate) {
    using P = Pack<T, VEC>;
    extern __shared__ __align__(16) unsigned char grad_smem[];
    const int lane = threadIdx.x & 31;
    P *ring = reinterpret_cast<P *>(grad_smem) + (threadIdx.x >> 5) * RING * 32 + lane;   // [RING][32]
    const int64_t item = blockIdx.x * static_cast<int64_t>(EMBED_THREADS / 32) + (threadIdx.x >> 5);
    dependents_may_launch();
    wait_for_prerequisites();
    if (item >= items) return;
    const int64_t c = static_cast<int64_t>(item % slabs) * (32 * VEC) + lane * VEC;
    const bool in = c < d;
    const uint32_t chunk = static_cast<uint32_t>(item / slabs);
    const uint64_t i0 = static_cast<uint64_t>(chunk) * L, i1 = i0 + L;
    auto key_at = [&](uint64_t i) { return i < n ? key[i] : V; };   // V: takes no part
    const uint32_t first = key_at(i0), last = key_at(i1 - 1);
    const uint32_t next0 = key_at(i1), next1 = key_at(i1 + L - 1);  // ends of the next chunk
    const uint32_t prev0 = i0 > 0 ? key[i0 - L] : 0xffffffffu;       // and of the one before
    const uint32_t prev1 = i0 > 0 ? key[i0 - 1] : 0xffffffffu;
    if (first >= V) return;
    const bool whole = first == last;
    // the segment that came in from the left: its part is ours only if it is long
    const bool came_in = first == prev1;
    const bool head_long = came_in && (whole || prev0 == first);
    const bool skip = came_in && !head_long;
    // the segment that goes on to the right
    const bool goes_on = last < V && next0 == last;
    const bool tail_long = goes_on && (whole || next1 == last);
    const int blocks = L / 32 * (goes_on && !tail_long ? 2 : 1);
    // 32 pairs at a time; taken: those of this warp (consecutive ones), starts:
    // the first ones of their segments
    struct Block { uint32_t k, p; unsigned taken, starts; };
    auto fetch = [&](int b, uint32_t k_before) {
        Block r{V, 0, 0, 0};
        if (b >= blocks) return r;
        const uint64_t i = i0 + b * 32 + lane;
        r.k = key_at(i);
        r.p = i < n ? pos[i] : 0;
        const bool take = r.k < V && (i < i1 ? !(skip && r.k == first) : r.k == last);
        uint32_t before = __shfl_up_sync(FULL_MASK, r.k, 1);
        if (lane == 0) before = k_before;
        r.taken = __ballot_sync(FULL_MASK, take);
        r.starts = __ballot_sync(FULL_MASK, take && r.k != before);
        return r;
    };
    int b = 0;
    Block now = fetch(0, V);
    while (now.taken == 0 && ++b < L / 32) now = fetch(b, V);   // skipped pairs
    if (now.taken == 0) return;
    const int j_first = __ffs(now.taken) - 1;
    now.starts &= ~(1u << j_first);
    Block next = fetch(b + 1, __shfl_sync(FULL_MASK, now.k, 31));
    auto rows_of = [&] {   // rows from `now` on, across the edge to `next`
        const int end = 32 - __clz(now.taken);
        return end == 32 ? 32 + __popc(next.taken) : end;
    };
    int m = rows_of();
    float acc[VEC] = {};
    uint32_t cur = __shfl_sync(FULL_MASK, now.k, j_first);
    bool in_part = head_long;   // the current segment came in from the left
    auto flush = [&](bool out_part) {
        if (!in_part && !out_part) {
            if (in) write_row<T, VEC>(gW + static_cast<int64_t>(cur) * d + c, acc, scale, accumulate);
        } else {
            float *to = part + (static_cast<int64_t>(chunk) * 2 + (in_part ? 0 : 1)) * d + c;
            if (in) store_f32<float, VEC>(to, acc);
            if (!in_part && c == 0) reinterpret_cast<uint2 *>(spanning)[1 + atomicAdd(spanning, 1u)] = make_uint2(chunk, cur);
        }
    };
    // starts the copies of rows j0 .. j0 + 7
    auto issue = [&](int j0) {
        P direct[BATCH];
#pragma unroll
        for (int a = 0; a < BATCH; ++a) {
            const int j = j0 + a;
            const uint32_t at0 = __shfl_sync(FULL_MASK, now.p, j & 31), at1 = __shfl_sync(FULL_MASK, next.p, j & 31);
            const T *src = g + static_cast<int64_t>(j < 32 ? at0 : at1) * d + c;
            if (!in || j >= m) continue;
            if (sizeof(P) >= 4) copy_async<sizeof(P)>(ring + j % RING * 32, src);
            else direct[a] = *reinterpret_cast<const P *>(src);
        }
        if (sizeof(P) >= 4) {
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
#pragma unroll
            for (int a = 0; a < BATCH; ++a)
                if (in && j0 + a < m) ring[(j0 + a) % RING * 32] = direct[a];
        }
    };
    issue(j_first);
    for (int j0 = j_first; j0 < m;) {
        issue(j0 + BATCH);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        const int j1 = j0 + BATCH < m ? j0 + BATCH : m;
#pragma unroll 4
        for (int j = j0; j < j1; ++j) {
            if ((j < 32 ? now.starts >> j : next.starts >> (j - 32)) & 1u) {
                flush(false);
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
                cur = __shfl_sync(FULL_MASK, j < 32 ? now.k : next.k, j & 31);
                in_part = false;
            }
            const P v = ring[j % RING * 32];
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] += to_f32(v.v[e]);
        }
        j0 += BATCH;
        if (j0 >= 32 && m > 32) {   // on to the next block; 32 is a multiple of the ring
            j0 -= 32;
            now = next;
            next = fetch(++b + 1, __shfl_sync(FULL_MASK, now.k, 31));
            m = rows_of();
        }
    }
    flush(tail_long && cur == last);
}

// Joins the parts of the long segments: a CTA per (segment, slab); its warps take every JOIN_WARPS-th chunk and the warps' sums are added
// in order.
constexpr int JOIN_WARPS = 16, JOIN_CTAS = 152 * 4;

template <typename T, int VEC>
__global__ void __launch_bounds__(JOIN_WARPS * 32)
    k_embed_join(const uint32_t *__restrict__ key, const float *__restrict__ part,
                 const uint32_t *__restrict__ spanning, T *__restrict__ gW, uint32_t n, int64_t d,
                 int L, int slabs, float scale, bool accumulate) {
    __shared__ float sum[JOIN_WARPS][32][VEC + 1];
    wait_for_prerequisites();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(spanning[0]) * slabs;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint2 entry = reinterpret_cast<const uint2 *>(spanning)[1 + item / slabs];
        const uint32_t c0 = entry.x, k = entry.y;
        const int64_t c = static_cast<int64_t>(item % slabs) * (32 * VEC) + lane * VEC;
        // its last chunk: the chunks after c0 that begin with k, counted by all threads
        uint32_t c1 = c0;
        for (int got = JOIN_WARPS * 32; got == JOIN_WARPS * 32; c1 += got) {
            const uint64_t i = (static_cast<uint64_t>(c1) + 1 + threadIdx.x) * L;
            got = __syncthreads_count(i < n && key[i] == k);
        }
        float acc[VEC] = {};
        if (c < d) {
#pragma unroll 8
            for (uint32_t q = c0 + w; q <= c1; q += JOIN_WARPS) {
                float v[VEC];
                load_f32<float, VEC>(part + (static_cast<int64_t>(q) * 2 + (q == c0 ? 1 : 0)) * d + c, v);
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[e] += v[e];
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[w][lane][e] = acc[e];
        __syncthreads();
        if (w == 0 && c < d) {
            for (int q = 1; q < JOIN_WARPS; ++q)
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[e] += sum[q][lane][e];
            write_row<T, VEC>(gW + static_cast<int64_t>(k) * d + c, acc, scale, accumulate);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host side
struct GradLayout {
    size_t key[2], pos[2], count, spanning, part, total;
};

GradLayout grad_layout(int64_t n, int64_t d) {
    GradLayout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const int64_t chunks = (n + MIN_CHUNK - 1) / MIN_CHUNK;
    for (int i = 0; i < 2; ++i) {
        l.key[i] = take(sizeof(uint32_t) * n);
        l.pos[i] = take(sizeof(uint32_t) * n);
    }
    l.count = take(sizeof(uint32_t) * SORT_CTAS * SORT_DIGITS);
    l.spanning = take(2 * sizeof(uint32_t) * (1 + chunks));
    l.part = take(sizeof(float) * chunks * 2 * d);
    l.total = at;
    return l;
}

int check_embedding(const void *ids, int ids_type, int dtype, int64_t n, int64_t V, int64_t d) {
    if (dtype != NRNN_F32 && dtype != NRNN_BF16) return NRNN_ERR_INVALID_ARG;
    if (ids_type != NRNN_I32 && ids_type != NRNN_I64) return NRNN_ERR_INVALID_ARG;
    if (n < 0 || V <= 0 || d <= 0 || (n > 0 && ids == nullptr)) return NRNN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(ids) % (ids_type == NRNN_I64 ? 8 : 4) != 0)
        return NRNN_ERR_INVALID_ARG;
    if (n > INT32_MAX || V >= INT32_MAX || d > (1 << 24)) return NRNN_ERR_UNSUPPORTED;
    return NRNN_OK;
}

template <typename T, int VEC>
cudaError_t lookup(const void *ids, int ids_type, const void *W, void *out, int64_t n, int64_t V,
                   int64_t d, int64_t pad, float scale, cudaStream_t stream) {
    const int slabs = static_cast<int>((d + 32 * VEC - 1) / (32 * VEC));
    const int64_t items = (n + GROUP_ROWS - 1) / GROUP_ROWS * slabs;
    const int64_t blocks = (items + EMBED_THREADS / 32 - 1) / (EMBED_THREADS / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(ids_type == NRNN_I64 ? k_embedding<T, VEC, int64_t> : k_embedding<T, VEC, int32_t>,
                            static_cast<unsigned>(blocks), EMBED_THREADS, 0, stream, ids,
                            static_cast<const T *>(W), static_cast<T *>(out), n, V, d, slabs, pad, scale);
}

template <typename T, int VEC>
cudaError_t gradient(const void *g, void *gW, const SortArgs &a, float *part, int64_t n, int64_t d,
                     float scale, bool accumulate, cudaStream_t stream) {
    constexpr int smem = EMBED_THREADS * RING * static_cast<int>(sizeof(Pack<T, VEC>));
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = once_per_device(configured, [](int) {
        return cudaFuncSetAttribute(k_embed_grad<T, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    const int slabs = static_cast<int>((d + 32 * VEC - 1) / (32 * VEC));
    // the chunks set the order of the sums: by the warps of aligned rows, whatever these are
    const int vec = vec_of(sizeof(T), d, 32, {});
    const int64_t full_slabs = (d + 32 * vec - 1) / (32 * vec);
    int L = MIN_CHUNK;
    while (L < MAX_CHUNK && (n + L - 1) / L * full_slabs > FEW_WARPS) L *= 2;
    const int64_t items = (n + L - 1) / L * slabs;
    const int64_t blocks = (items + EMBED_THREADS / 32 - 1) / (EMBED_THREADS / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    e = launch_dependent(k_embed_grad<T, VEC>, static_cast<unsigned>(blocks), EMBED_THREADS, smem, stream,
                         a.kin, a.pin, static_cast<const T *>(g), static_cast<T *>(gW), part,
                         a.spanning, a.n, a.V, d, L, slabs, items, scale, accumulate);
    if (e != cudaSuccess || n <= L) return e;
    const int64_t most = n / L * slabs;
    return launch_dependent(k_embed_join<T, VEC>, static_cast<unsigned>(most < JOIN_CTAS ? most : JOIN_CTAS),
                            JOIN_WARPS * 32, 0, stream, a.kin, part, a.spanning,
                            static_cast<T *>(gW), a.n, d, L, slabs, scale, accumulate);
}

}  // namespace
}  // namespace nrnn

using namespace nrnn;

extern "C" {

int nrnn_embedding(const void *ids, int ids_type, const void *W, int dtype, int64_t n, int64_t V,
                   int64_t d, int64_t padding_id, float scale, void *out, void *stream) {
    const int st = check_embedding(ids, ids_type, dtype, n, V, d);
    if (st != NRNN_OK) return st;
    if (n == 0) return NRNN_OK;
    const int elem = dtype == NRNN_BF16 ? 2 : 4;
    if (W == nullptr || out == nullptr) return NRNN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(W) | reinterpret_cast<uintptr_t>(out)) % elem != 0)
        return NRNN_ERR_INVALID_ARG;
    if (padding_id < 0 || padding_id >= V) padding_id = -1;   // none
    const int vec = vec_of(elem, d, 32, {W, out});
    const cudaError_t e = NRNN_BY_WIDTH(dtype, vec, lookup, ids, ids_type, W, out, n, V, d,
                                        padding_id, scale, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

size_t nrnn_embedding_backward_workspace_bytes(int64_t n, int64_t V, int64_t d) {
    if (n < 0 || V <= 0 || d <= 0 || n > INT32_MAX || V >= INT32_MAX || d > (1 << 24)) return 0;
    return grad_layout(n, d).total;
}

int nrnn_embedding_backward(const void *ids, int ids_type, const void *g, int dtype, int64_t n,
                            int64_t V, int64_t d, int64_t padding_id, float scale, int accumulate,
                            void *gW, void *workspace, size_t ws_bytes, void *stream) {
    const int st = check_embedding(ids, ids_type, dtype, n, V, d);
    if (st != NRNN_OK) return st;
    const int elem = dtype == NRNN_BF16 ? 2 : 4;
    if (gW == nullptr || (n > 0 && g == nullptr)) return NRNN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(gW)) % elem != 0)
        return NRNN_ERR_INVALID_ARG;
    const GradLayout l = grad_layout(n, d);
    if (workspace == nullptr || ws_bytes < l.total || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return NRNN_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n == 0) {
        if (accumulate) return NRNN_OK;
        return cudaMemsetAsync(gW, 0, static_cast<size_t>(V) * d * elem, s) == cudaSuccess
                   ? NRNN_OK : NRNN_ERR_CUDA;
    }
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    SortArgs a{};
    a.ids = ids;
    a.n = static_cast<uint32_t>(n);
    a.V = static_cast<uint32_t>(V);
    a.pad = padding_id;
    uint32_t *const key[2] = {reinterpret_cast<uint32_t *>(ws + l.key[0]),
                              reinterpret_cast<uint32_t *>(ws + l.key[1])};
    uint32_t *const pos[2] = {reinterpret_cast<uint32_t *>(ws + l.pos[0]),
                              reinterpret_cast<uint32_t *>(ws + l.pos[1])};
    a.count = reinterpret_cast<uint32_t *>(ws + l.count);
    a.spanning = reinterpret_cast<uint32_t *>(ws + l.spanning);
    int key_bits = 1;
    while ((static_cast<int64_t>(1) << key_bits) <= V) ++key_bits;   // keys 0 .. V
    const int passes = (key_bits + SORT_MAX_BITS - 1) / SORT_MAX_BITS;
    a.bits = (key_bits + passes - 1) / passes;
    // the sort's launches clear gW, in whole 16-byte pieces but for its ends
    const size_t gw_bytes = static_cast<size_t>(V) * d * elem;
    unsigned char *to = static_cast<unsigned char *>(gW);
    size_t head = (16 - reinterpret_cast<uintptr_t>(gW) % 16) % 16;
    if (head > gw_bytes) head = gw_bytes;
    const int64_t clear16 = accumulate ? 0 : static_cast<int64_t>((gw_bytes - head) / 16);
    if (!accumulate) {
        a.end_bytes[0] = static_cast<int>(head);
        a.end_bytes[1] = static_cast<int>((gw_bytes - head) % 16);
        a.ends[0] = to;
        a.ends[1] = to + gw_bytes - a.end_bytes[1];
    }
    cudaError_t e = ids_type == NRNN_I64 ? sort_ids<int64_t>(a, key, pos, passes, to + head, clear16, accumulate == 0, s)
                                         : sort_ids<int32_t>(a, key, pos, passes, to + head, clear16, accumulate == 0, s);
    if (e != cudaSuccess) return NRNN_ERR_CUDA;
    a.kin = key[1];   // the sorted pairs
    a.pin = pos[1];
    const int vec = vec_of(elem, d, 32, {g, gW});
    e = NRNN_BY_WIDTH(dtype, vec, gradient, g, gW, a, reinterpret_cast<float *>(ws + l.part), n, d,
                      scale, accumulate != 0, s);
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

}  // extern "C"
