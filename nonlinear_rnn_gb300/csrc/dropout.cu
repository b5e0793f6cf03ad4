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
    uint64_t limit;            // keep a word >= limit; 2^32: none
    float scale;
};

constexpr int DROP_THREADS = 256;

// VEC elements a thread: 16 bytes where all tensors are aligned to them, else one
template <typename T, int VEC>
__global__ void __launch_bounds__(DROP_THREADS) k_dropout(const DropArgs a) {
    dependents_may_launch();
    wait_for_prerequisites();
    const uint64_t seed = a.seed_at != nullptr ? *a.seed_at : a.seed;
    const uint2 key = make_uint2(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
    const T *x = static_cast<const T *>(a.x), *residual = static_cast<const T *>(a.residual);
    T *out = static_cast<T *>(a.out);
    constexpr int GROUP = VEC < 4 ? 4 : VEC;
    const int64_t groups = (a.n + GROUP - 1) / GROUP;
    const int64_t step = static_cast<int64_t>(gridDim.x) * DROP_THREADS;
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * DROP_THREADS + threadIdx.x; g < groups; g += step) {
        const int64_t e0 = g * GROUP;
        uint32_t word[GROUP];
#pragma unroll
        for (int q = 0; q < GROUP / 4; ++q) {
            const uint4 w = philox(static_cast<uint64_t>(e0 / 4 + q), a.offset, key);
            word[4 * q] = w.x;
            word[4 * q + 1] = w.y;
            word[4 * q + 2] = w.z;
            word[4 * q + 3] = w.w;
        }
        if (VEC > 1 && e0 + GROUP <= a.n) {
            float v[GROUP], r[GROUP] = {};
            load_f32<T, GROUP>(x + e0, v);
            if (residual != nullptr) load_f32<T, GROUP>(residual + e0, r);
#pragma unroll
            for (int e = 0; e < GROUP; ++e) v[e] = word[e] >= a.limit ? fmaf(v[e], a.scale, r[e]) : r[e];
            store_f32<T, GROUP>(out + e0, v);
        } else {
#pragma unroll
            for (int e = 0; e < GROUP; ++e)
                if (e0 + e < a.n) {
                    const float r = residual != nullptr ? to_f32(residual[e0 + e]) : 0.f;
                    out[e0 + e] = from_f32<T>(word[e] >= a.limit ? fmaf(to_f32(x[e0 + e]), a.scale, r) : r);
                }
        }
    }
}

template <typename T>
cudaError_t dropout(const DropArgs &a, cudaStream_t s) {
    constexpr int VEC = 16 / sizeof(T);
    const bool wide = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                        reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    const int64_t groups = (a.n + (wide ? VEC : 4) - 1) / (wide ? VEC : 4), want = (groups + DROP_THREADS - 1) / DROP_THREADS;
    const unsigned blocks = static_cast<unsigned>(want < 152 * 64 ? want : 152 * 64);
    return wide ? launch_dependent(k_dropout<T, VEC>, blocks, DROP_THREADS, 0, s, a)
                : launch_dependent(k_dropout<T, 1>, blocks, DROP_THREADS, 0, s, a);
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
    a.limit = static_cast<uint64_t>(std::nearbyint(p * 4294967296.0));
    a.scale = p < 1.0 ? static_cast<float>(1.0 / (1.0 - p)) : 0.f;
    const cudaError_t e = dtype == NRNN_BF16 ? dropout<__nv_bfloat16>(a, static_cast<cudaStream_t>(stream))
                                             : dropout<float>(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}
