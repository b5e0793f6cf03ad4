// Dropout from a counter-based generator: the mask is made again wherever it is
// needed and never stored.
//
//   y_e = residual_e + x_e keep_e / (1 - p),  keep_e = word(e) >= round(p 2^32)
//
// word(e) is the (e mod 4)-th word of the Philox 4x32 generator of ten rounds
// (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011) with the counter {e / 4 low, e / 4 high, offset low, offset high} and the
// key {seed low, seed high}.  The gradient with respect to x is the same call on
// the gradient.  What is dropped is zero whatever x holds.
//
// 2 or 3 values an element through HBM; beside them ten rounds of two wide products for
// four elements, which take most of the issue slots: 262144 x 1024 bf16 with residual 273 us
// (0.87 of HBM's measured rate; with four rounds it would be 0.94).  A group's loads are
// under way while its words are made; two groups at a time were slower (317), as was a
// threshold of 64 bits, which holds p = 1 too (300).
#include <cmath>

#include "../../include/nrnn.h"
#include "nrnn_internal.h"
#include "rows.cuh"

namespace nrnn {
namespace {

__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t offset, uint2 key) {
    uint4 c = make_uint4(static_cast<uint32_t>(block), static_cast<uint32_t>(block >> 32),
                         static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32));
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c.x, p1 = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
        c = make_uint4(static_cast<uint32_t>(p1 >> 32) ^ c.y ^ key.x, static_cast<uint32_t>(p1),
                       static_cast<uint32_t>(p0 >> 32) ^ c.w ^ key.y, static_cast<uint32_t>(p0));
        key.x += 0x9E3779B9u;
        key.y += 0xBB67AE85u;
    }
    return c;
}

struct DropArgs {
    const void *x, *residual;
    void *out;
    int64_t n;
    uint64_t seed, offset;
    const uint64_t *seed_at;   // device; null: seed
    uint32_t limit;            // keep a word >= limit
    float scale;
};

constexpr int DROP_THREADS = 256;

__device__ __forceinline__ float dropped(uint32_t word, const DropArgs &a, float x, float r) {
    return word >= a.limit ? fmaf(x, a.scale, r) : r;
}

// A thread takes groups of 16 bytes where all tensors are aligned to them (WIDE), else of
// four elements, whose words one Philox block gives.
template <typename T, bool WIDE, bool RESIDUAL>
__global__ void __launch_bounds__(DROP_THREADS) k_dropout(const DropArgs a) {
    constexpr int GROUP = WIDE ? 16 / sizeof(T) : 4;
    dependents_may_launch();
    wait_for_prerequisites();
    const uint64_t seed = a.seed_at != nullptr ? *a.seed_at : a.seed;
    const uint2 key = make_uint2(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
    const T *x = static_cast<const T *>(a.x), *residual = static_cast<const T *>(a.residual);
    T *out = static_cast<T *>(a.out);
    const int64_t whole = WIDE ? a.n / GROUP : 0;   // groups that are loaded and stored at once
    const int64_t threads = static_cast<int64_t>(gridDim.x) * DROP_THREADS;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * DROP_THREADS + threadIdx.x;
    for (int64_t g = first; g < whole; g += threads) {
        Pack<T, GROUP> r{};
        const Pack<T, GROUP> v = *reinterpret_cast<const Pack<T, GROUP> *>(x + g * GROUP);   // under way while the words are made
        if (RESIDUAL) r = *reinterpret_cast<const Pack<T, GROUP> *>(residual + g * GROUP);
        float o[GROUP];
#pragma unroll
        for (int q = 0; q < GROUP; q += 4) {
            const uint4 w4 = philox(static_cast<uint64_t>(g * (GROUP / 4) + q / 4), a.offset, key);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) o[q + e] = dropped(w[e], a, to_f32(v.v[q + e]), to_f32(r.v[q + e]));
        }
        store_f32<T, GROUP>(out + g * GROUP, o);
    }
    // the rest, four elements at a time (a whole group is a multiple of four)
    const int64_t quads = (a.n + 3) / 4;
    for (int64_t b = whole * (GROUP / 4) + first; b < quads; b += threads) {
        const uint4 w4 = philox(static_cast<uint64_t>(b), a.offset, key);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        float v[4], r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = b * 4 + e < a.n;
            v[e] = in ? to_f32(x[b * 4 + e]) : 0.f;
            r[e] = in && RESIDUAL ? to_f32(residual[b * 4 + e]) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (b * 4 + e < a.n) out[b * 4 + e] = from_f32<T>(dropped(w[e], a, v[e], r[e]));
    }
}

template <typename T>
cudaError_t dropout(const DropArgs &a, cudaStream_t s) {
    const bool wide = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                        reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    const int64_t per_block = DROP_THREADS * (wide ? 16 / static_cast<int64_t>(sizeof(T)) : 4);
    const int64_t want = (a.n + per_block - 1) / per_block;
    const unsigned blocks = static_cast<unsigned>(want < 152 * 64 ? want : 152 * 64);
    if (a.residual != nullptr)
        return wide ? launch_dependent(k_dropout<T, true, true>, blocks, DROP_THREADS, 0, s, a)
                    : launch_dependent(k_dropout<T, false, true>, blocks, DROP_THREADS, 0, s, a);
    return wide ? launch_dependent(k_dropout<T, true, false>, blocks, DROP_THREADS, 0, s, a)
                : launch_dependent(k_dropout<T, false, false>, blocks, DROP_THREADS, 0, s, a);
}

}  // namespace
}  // namespace nrnn

using namespace nrnn;

extern "C" int nrnn_dropout(const void *x, int dtype, int64_t n, double p, uint64_t seed, const uint64_t *seed_device,
                            uint64_t offset, const void *residual, void *out, void *stream) {
    if (dtype != NRNN_F32 && dtype != NRNN_BF16) return NRNN_ERR_INVALID_ARG;
    if (n < 0 || !(p >= 0.0 && p <= 1.0)) return NRNN_ERR_INVALID_ARG;
    if (n > (1ll << 48)) return NRNN_ERR_UNSUPPORTED;
    if (n == 0) return NRNN_OK;
    const uintptr_t elem = dtype == NRNN_BF16 ? 2 : 4, bytes = elem * n;
    const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ra = reinterpret_cast<uintptr_t>(residual),
                    oa = reinterpret_cast<uintptr_t>(out);
    if (x == nullptr || out == nullptr || (xa | ra | oa) % elem != 0 || reinterpret_cast<uintptr_t>(seed_device) % 8 != 0)
        return NRNN_ERR_INVALID_ARG;
    // out may be x or residual, but not reach into either from another place
    for (const uintptr_t in : {xa, ra})
        if (in != 0 && in != oa && in < oa + bytes && oa < in + bytes) return NRNN_ERR_INVALID_ARG;
    DropArgs a{};
    a.x = x; a.residual = residual; a.out = out; a.n = n;
    a.seed = seed; a.seed_at = seed_device; a.offset = offset;
    const double limit = std::nearbyint(p * 4294967296.0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (limit >= 4294967296.0) {   // nothing is kept
        if (residual == nullptr) e = cudaMemsetAsync(out, 0, bytes, s);
        else if (out != residual) e = cudaMemcpyAsync(out, residual, bytes, cudaMemcpyDeviceToDevice, s);
        return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
    }
    a.limit = static_cast<uint32_t>(limit);
    a.scale = static_cast<float>(1.0 / (1.0 - p));
    e = dtype == NRNN_BF16 ? dropout<__nv_bfloat16>(a, s)
                                             : dropout<float>(a, s);
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}
