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
// radix sort, and the sums follow the sorted order in fixed groups of 32.
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
constexpr int EMBED_THREADS = 256;

template <typename Id> __device__ __forceinline__ int64_t id_at(const void *ids, int64_t i) {
    return static_cast<int64_t>(static_cast<const Id *>(ids)[i]);
}

// ------------------------------------------------------------------ the lookup
// A warp copies one slab of GROUP_ROWS rows, all loads before the first store.
// An id outside [0, V) that is not the padding id gives a row of NaN.
template <typename T, int VEC, typename Id>
__global__ void __launch_bounds__(EMBED_THREADS)
    k_embedding(const void *__restrict__ ids, const T *__restrict__ W, T *__restrict__ out,
                int64_t n, int64_t V, int64_t d, int slabs, int64_t pad, float scale) {
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
// Stable least-significant-digit radix sort of (id, position) by one cluster of
// CTAs, all passes in one launch: the digit counts are exchanged through
// distributed shared memory between two cluster barriers, where separate
// launches would cost several microseconds each.  Every warp owns a contiguous
// range of the input, so ranks follow (CTA, warp, step, lane) = input order.
// Ids that take no part (padding, out of range) get the key V and sort last.
constexpr int SORT_CTAS = 8;
constexpr int SORT_THREADS = 1024, SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_MAX_BITS = 9, SORT_DIGITS = 1 << SORT_MAX_BITS;
constexpr size_t SORT_SMEM = sizeof(uint32_t) * SORT_DIGITS * (SORT_WARPS + 2);

struct SortBuffers {
    uint32_t *key[2], *pos[2];   // the sorted pairs end in [1]
    uint8_t *present;            // V flags: the id occurs (null: not wanted)
    uint32_t *spanning;          // count of the list of segments that span chunks
};

template <typename Id>
__global__ void __cluster_dims__(SORT_CTAS, 1, 1) __launch_bounds__(SORT_THREADS)
    k_sort_ids(const void *ids, uint32_t n, uint32_t V, int64_t pad, SortBuffers b, int passes,
               int bits) {
    extern __shared__ uint32_t sort_smem[];
    uint32_t *cnt = sort_smem;                              // [SORT_WARPS][SORT_DIGITS]
    uint32_t *total = cnt + SORT_WARPS * SORT_DIGITS;       // [SORT_DIGITS] this CTA's counts
    uint32_t *base = total + SORT_DIGITS;                   // [SORT_DIGITS] first place of a digit
    __shared__ uint32_t warp_sum[SORT_DIGITS / 32];
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t r = cluster.block_rank();
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const uint32_t mask = (1u << bits) - 1u;
    // steps of 32 pairs per warp
    const uint32_t steps = (n + SORT_CTAS * SORT_THREADS - 1) / (SORT_CTAS * SORT_THREADS);
    const uint64_t w0 = (static_cast<uint64_t>(r) * SORT_WARPS + w) * steps * 32;

    if (b.present != nullptr)
        for (uint32_t i = r * SORT_THREADS + tid; i < V; i += SORT_CTAS * SORT_THREADS)
            b.present[i] = 0;
    if (r == 0 && tid == 0) *b.spanning = 0;

    for (int p = 0; p < passes; ++p) {
        const int shift = p * bits;
        // the last pass writes [1]
        const int to = (passes - 1 - p) & 1 ? 0 : 1;
        const uint32_t *kin = b.key[to ^ 1], *pin = b.pos[to ^ 1];
        uint32_t *kout = b.key[to], *pout = b.pos[to];
        auto key_at = [&](uint64_t i) -> uint32_t {
            if (i >= n) return 0xffffffffu;
            if (p > 0) return __ldcg(kin + i);
            const int64_t id = id_at<Id>(ids, i);
            return id >= 0 && id < V && id != pad ? static_cast<uint32_t>(id) : V;
        };
        uint32_t *mine = cnt + w * SORT_DIGITS;
        for (int i = tid; i < SORT_WARPS * SORT_DIGITS; i += SORT_THREADS) cnt[i] = 0;
        __syncthreads();
        for (uint32_t s = 0; s < steps; ++s) {
            const uint64_t i = w0 + static_cast<uint64_t>(s) * 32 + lane;
            const uint32_t k = key_at(i);
            const uint32_t digit = i < n ? (k >> shift) & mask : 0xffffffffu;
            const unsigned peers = __match_any_sync(FULL_MASK, digit);
            if (i < n && lane == __ffs(peers) - 1) mine[digit] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        if (tid < SORT_DIGITS) {
            uint32_t run = 0;
#pragma unroll 8
            for (int v = 0; v < SORT_WARPS; ++v) {
                const uint32_t c = cnt[v * SORT_DIGITS + tid];
                cnt[v * SORT_DIGITS + tid] = run;
                run += c;
            }
            total[tid] = run;
        }
        cluster.sync();
        uint32_t before = 0, all = 0;
        if (tid < SORT_DIGITS) {
            for (uint32_t c = 0; c < SORT_CTAS; ++c) {
                const uint32_t t = *cluster.map_shared_rank(total + tid, c);
                before += c < r ? t : 0;
                all += t;
            }
        }
        // exclusive scan of `all` over the digits (the first 16 warps)
        uint32_t incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(FULL_MASK, incl, o);
            if (lane >= o) incl += t;
        }
        if (tid < SORT_DIGITS && lane == 31) warp_sum[w] = incl;
        __syncthreads();
        if (tid < SORT_DIGITS) {
            uint32_t lower = 0;
            for (int v = 0; v < w; ++v) lower += warp_sum[v];
            base[tid] = lower + incl - all + before;
        }
        __syncthreads();
        for (int i = tid; i < SORT_WARPS * SORT_DIGITS; i += SORT_THREADS)
            cnt[i] += base[i & (SORT_DIGITS - 1)];
        __syncthreads();
        for (uint32_t s = 0; s < steps; ++s) {
            const uint64_t i = w0 + static_cast<uint64_t>(s) * 32 + lane;
            const uint32_t k = key_at(i);
            const uint32_t digit = i < n ? (k >> shift) & mask : 0xffffffffu;
            const unsigned peers = __match_any_sync(FULL_MASK, digit);
            const uint32_t first = i < n ? mine[digit] : 0;
            __syncwarp();
            if (i < n) {
                const uint32_t at = first + __popc(peers & ((1u << lane) - 1u));
                kout[at] = k;
                pout[at] = p > 0 ? __ldcg(pin + i) : static_cast<uint32_t>(i);
                if (lane == __ffs(peers) - 1) mine[digit] = first + __popc(peers);
            }
            __syncwarp();
        }
        cluster.sync();   // this pass's pairs are visible; `total` is free again
    }
    if (b.present != nullptr) {
        const uint32_t *keys = b.key[1];
        for (uint64_t i = r * SORT_THREADS + tid; i < n; i += SORT_CTAS * SORT_THREADS) {
            const uint32_t k = __ldcg(keys + i);
            if (k < V && (i == 0 || __ldcg(keys + i - 1) != k)) b.present[k] = 1;
        }
    }
}

// ---------------------------------------------------------------- the gradient
// A warp sums one slab of a chunk of 32 consecutive sorted pairs, eight rows of
// loads in flight.  A segment (the pairs of one id) inside the chunk is written
// at once; one that crosses a chunk's edge leaves fp32 partial sums: slot 0 of a
// chunk for the segment that came in from the left, slot 1 for one that begins
// here and goes on.  Those are joined in order by k_embed_join.
constexpr int CHUNK = 32;

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

template <typename T, int VEC>
__global__ void __launch_bounds__(EMBED_THREADS)
    k_embed_grad(const uint32_t *__restrict__ key, const uint32_t *__restrict__ pos,
                 const uint8_t *__restrict__ present, const T *__restrict__ g, T *__restrict__ gW,
                 float *__restrict__ part, uint32_t *__restrict__ spanning, uint32_t n, uint32_t V,
                 int64_t d, int slabs, int64_t chunk_items, int64_t items, float scale,
                 bool accumulate) {
    const int lane = threadIdx.x & 31;
    int64_t item = blockIdx.x * static_cast<int64_t>(EMBED_THREADS / 32) + (threadIdx.x >> 5);
    if (item >= items) return;
    const bool zero = item >= chunk_items;
    if (zero) item -= chunk_items;
    const int64_t c = static_cast<int64_t>(item % slabs) * (32 * VEC) + lane * VEC;
    const bool in = c < d;
    if (zero) {   // rows of ids that do not occur
        const int64_t v0 = item / slabs * 32;
        const bool absent = v0 + lane < V && present[v0 + lane] == 0;
        unsigned todo = __ballot_sync(FULL_MASK, absent);
        const float none[VEC] = {};
        while (todo != 0) {
            const int j = __ffs(todo) - 1;
            todo &= todo - 1;
            if (in) store_f32<T, VEC>(gW + (v0 + j) * d + c, none);
        }
        return;
    }
    const uint32_t chunk = static_cast<uint32_t>(item / slabs);
    const uint64_t i0 = static_cast<uint64_t>(chunk) * CHUNK;
    const uint32_t k_lane = i0 + lane < n ? key[i0 + lane] : V;
    const uint32_t p_lane = i0 + lane < n ? pos[i0 + lane] : 0;
    const uint32_t k_prev = i0 > 0 ? key[i0 - 1] : 0xffffffffu;
    const uint32_t k_next = i0 + CHUNK < n ? key[i0 + CHUNK] : V;
    const int m = __popc(__ballot_sync(FULL_MASK, k_lane < V));   // valid pairs come first
    float acc[VEC] = {};
    uint32_t cur = __shfl_sync(FULL_MASK, k_lane, 0);
    bool began = cur != k_prev;   // the current segment begins in this chunk
    auto flush = [&](bool ended) {
        if (began && ended) {
            if (in) write_row<T, VEC>(gW + static_cast<int64_t>(cur) * d + c, acc, scale, accumulate);
        } else {
            float *to = part + (static_cast<int64_t>(chunk) * 2 + (began ? 1 : 0)) * d + c;
            if (in) store_f32<float, VEC>(to, acc);
            if (began && c == 0) spanning[1 + atomicAdd(spanning, 1u)] = chunk;
        }
    };
    constexpr int AHEAD = 8;
    for (int j0 = 0; j0 < m; j0 += AHEAD) {
        float v[AHEAD][VEC];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const uint32_t at = __shfl_sync(FULL_MASK, p_lane, (j0 + a) & 31);
            if (in && j0 + a < m) load_f32<T, VEC>(g + static_cast<int64_t>(at) * d + c, v[a]);
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            if (j0 + a >= m) break;
            const uint32_t k = __shfl_sync(FULL_MASK, k_lane, (j0 + a) & 31);
            if (k != cur) {
                flush(true);
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
                cur = k;
                began = true;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] += v[a][e];
        }
    }
    if (m > 0) flush(k_next != cur);
}

// Joins the partial sums of the segments that span chunks: a CTA per (segment,
// slab); its warps take every JOIN_WARPS-th chunk and the warps' sums are added
// in order.
constexpr int JOIN_WARPS = 16;

template <typename T, int VEC>
__global__ void __launch_bounds__(JOIN_WARPS * 32)
    k_embed_join(const uint32_t *__restrict__ key, const float *__restrict__ part,
                 const uint32_t *__restrict__ spanning, T *__restrict__ gW, uint32_t n, int64_t d,
                 int slabs, float scale, bool accumulate) {
    __shared__ float sum[JOIN_WARPS][32][VEC + 1];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(spanning[0]) * slabs;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t c0 = spanning[1 + item / slabs];
        const int64_t c = static_cast<int64_t>(item % slabs) * (32 * VEC) + lane * VEC;
        const uint32_t k = key[static_cast<uint64_t>(c0) * CHUNK + CHUNK - 1];
        // first pair after the segment
        uint64_t lo = static_cast<uint64_t>(c0 + 1) * CHUNK, hi = n;
        while (lo < hi) {
            const uint64_t mid = (lo + hi) / 2;
            if (key[mid] == k) lo = mid + 1; else hi = mid;
        }
        const uint32_t c1 = static_cast<uint32_t>((lo - 1) / CHUNK);   // its last chunk
        float acc[VEC] = {};
        if (c < d) {
#pragma unroll 4
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
    size_t key[2], pos[2], present, spanning, part, total;
};

GradLayout grad_layout(int64_t n, int64_t V, int64_t d) {
    GradLayout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const int64_t chunks = (n + CHUNK - 1) / CHUNK;
    for (int i = 0; i < 2; ++i) {
        l.key[i] = take(sizeof(uint32_t) * n);
        l.pos[i] = take(sizeof(uint32_t) * n);
    }
    l.present = take(V);
    l.spanning = take(sizeof(uint32_t) * (1 + chunks));
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
    auto kernel = ids_type == NRNN_I64 ? k_embedding<T, VEC, int64_t> : k_embedding<T, VEC, int32_t>;
    kernel<<<static_cast<unsigned>(blocks), EMBED_THREADS, 0, stream>>>(
        ids, static_cast<const T *>(W), static_cast<T *>(out), n, V, d, slabs, pad, scale);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t gradient(const void *g, void *gW, const SortBuffers &b, float *part, int64_t n,
                     int64_t V, int64_t d, float scale, bool accumulate, cudaStream_t stream) {
    const int slabs = static_cast<int>((d + 32 * VEC - 1) / (32 * VEC));
    const int64_t chunk_items = (n + CHUNK - 1) / CHUNK * slabs;
    const int64_t items = chunk_items + (accumulate ? 0 : (V + 31) / 32 * slabs);
    const int64_t blocks = (items + EMBED_THREADS / 32 - 1) / (EMBED_THREADS / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    k_embed_grad<T, VEC><<<static_cast<unsigned>(blocks), EMBED_THREADS, 0, stream>>>(
        b.key[1], b.pos[1], b.present, static_cast<const T *>(g), static_cast<T *>(gW), part,
        b.spanning, static_cast<uint32_t>(n), static_cast<uint32_t>(V), d, slabs, chunk_items,
        items, scale, accumulate);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || n <= CHUNK) return e;
    const int64_t most = (n / CHUNK) * slabs;
    k_embed_join<T, VEC><<<static_cast<unsigned>(most < 608 ? most : 608), JOIN_WARPS * 32, 0, stream>>>(
        b.key[1], part, b.spanning, static_cast<T *>(gW), static_cast<uint32_t>(n), d, slabs,
        scale, accumulate);
    return cudaGetLastError();
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
    return grad_layout(n, V, d).total;
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
    const GradLayout l = grad_layout(n, V, d);
    if (workspace == nullptr || ws_bytes < l.total || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return NRNN_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n == 0) {
        if (accumulate) return NRNN_OK;
        return cudaMemsetAsync(gW, 0, static_cast<size_t>(V) * d * elem, s) == cudaSuccess
                   ? NRNN_OK : NRNN_ERR_CUDA;
    }
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    SortBuffers b;
    for (int i = 0; i < 2; ++i) {
        b.key[i] = reinterpret_cast<uint32_t *>(ws + l.key[i]);
        b.pos[i] = reinterpret_cast<uint32_t *>(ws + l.pos[i]);
    }
    b.present = accumulate ? nullptr : ws + l.present;
    b.spanning = reinterpret_cast<uint32_t *>(ws + l.spanning);
    int key_bits = 1;
    while ((static_cast<int64_t>(1) << key_bits) <= V) ++key_bits;   // keys 0 .. V
    const int passes = (key_bits + SORT_MAX_BITS - 1) / SORT_MAX_BITS;
    const int bits = (key_bits + passes - 1) / passes;
    auto sort = ids_type == NRNN_I64 ? k_sort_ids<int64_t> : k_sort_ids<int32_t>;
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = once_per_device(configured, [](int) {
        cudaError_t r = cudaFuncSetAttribute(k_sort_ids<int64_t>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(SORT_SMEM));
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(k_sort_ids<int32_t>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(SORT_SMEM));
        return r;
    });
    if (e != cudaSuccess) return NRNN_ERR_CUDA;
    sort<<<SORT_CTAS, SORT_THREADS, SORT_SMEM, s>>>(ids, static_cast<uint32_t>(n),
                                                    static_cast<uint32_t>(V), padding_id, b, passes,
                                                    bits);
    e = cudaGetLastError();
    if (e != cudaSuccess) return NRNN_ERR_CUDA;
    const int vec = vec_of(elem, d, 32, {g, gW});
    e = NRNN_BY_WIDTH(dtype, vec, gradient, g, gW, b, reinterpret_cast<float *>(ws + l.part), n, V,
                      d, scale, accumulate != 0, s);
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

}  // extern "C"
