// Gated feed-forward block and its gradient.
//
//   a = x Wg^T, b = x Wu^T, m = silu(a) b, y = m Wo^T        W_in = [Wg; Wu]
//   gm = g Wo, ga = gm b silu'(a), gb = gm silu(a)
//   gx = [ga gb] W_in, gW_in = [ga gb]^T x, gW_out = g^T m
//
// 6 n d f operations forward and 12 n d f backward.
#include "../../include/nrnn.h"
#include "nrnn_internal.h"
#include "rows.cuh"

namespace nrnn {
namespace {

constexpr int TILE = 64, DEEP = 16;

struct Product {
    const void *A, *B;
    int64_t a_row, a_k, b_row, b_k;   // strides of a row and of an inner element
    int64_t M, N, K;
    void *out;
    int64_t pitch;
    bool add;
};

// out(m, n) = sum_k A(m, k) B(n, k), fp32 sums; 64 x 64 tiles, 4 x 4 a thread
template <typename T, typename O>
__global__ void __launch_bounds__(256) k_product(const Product p) {
    __shared__ float a[DEEP][TILE + 1], b[DEEP][TILE + 1];
    const T *A = static_cast<const T *>(p.A), *B = static_cast<const T *>(p.B);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * TILE;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * TILE; m0 < p.M; m0 += static_cast<int64_t>(gridDim.y) * TILE) {
        float c[4][4] = {};
        for (int64_t k0 = 0; k0 < p.K; k0 += DEEP) {
            for (int i = threadIdx.x; i < TILE * DEEP; i += 256) {
                const bool along_k = p.a_k == 1;
                const int r = along_k ? i / DEEP : i % TILE, k = along_k ? i % DEEP : i / TILE;
                a[k][r] = m0 + r < p.M && k0 + k < p.K ? to_f32(A[(m0 + r) * p.a_row + (k0 + k) * p.a_k]) : 0.f;
            }
            for (int i = threadIdx.x; i < TILE * DEEP; i += 256) {
                const bool along_k = p.b_k == 1;
                const int r = along_k ? i / DEEP : i % TILE, k = along_k ? i % DEEP : i / TILE;
                b[k][r] = n0 + r < p.N && k0 + k < p.K ? to_f32(B[(n0 + r) * p.b_row + (k0 + k) * p.b_k]) : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < DEEP; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[i][j] = fmaf(a[k][ty * 4 + i], b[k][tx + 16 * j], c[i][j]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
                if (m < p.M && n < p.N) {
                    O *o = static_cast<O *>(p.out) + m * p.pitch + n;
                    *o = from_f32<O>(p.add ? to_f32(*o) + c[i][j] : c[i][j]);
                }
            }
    }
}

__device__ __forceinline__ float sigmoid_of(float x) { return rcp_approx(1.f + ex2_approx(-LOG2E * x)); }

// a, b as kept for the gradient, m from them unrounded
template <typename T>
__global__ void __launch_bounds__(256) k_gate(const float *a, const float *b, T *ka, T *kb, T *m, int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const float x = a[i];
        ka[i] = from_f32<T>(x);
        kb[i] = from_f32<T>(b[i]);
        m[i] = from_f32<T>(x * sigmoid_of(x) * b[i]);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_gate_back(const T *a, const T *b, const float *gm, T *ga, T *gb, int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const float x = to_f32(a[i]), s = sigmoid_of(x), g = gm[i];
        ga[i] = from_f32<T>(g * to_f32(b[i]) * s * fmaf(x, 1.f - s, 1.f));
        gb[i] = from_f32<T>(g * x * s);
    }
}

template <typename T> __global__ void __launch_bounds__(256) k_round(const float *in, T *out, int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
        out[i] = from_f32<T>(in[i]);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Call {
    const void *x, *W_in, *W_out;
    int dtype;
    int64_t n, d, f;
    cudaStream_t stream;
};

template <typename T, typename O>
cudaError_t product(const Call &c, const void *A, int64_t a_row, int64_t a_k, const void *B, int64_t b_row, int64_t b_k,
                    int64_t M, int64_t N, int64_t K, O *out, int64_t pitch, bool add = false) {
    if (M == 0 || N == 0) return cudaSuccess;
    const Product p{A, B, a_row, a_k, b_row, b_k, M, N, K, out, pitch, add};
    const int64_t rows = (M + TILE - 1) / TILE;
    k_product<T, O><<<dim3(static_cast<unsigned>((N + TILE - 1) / TILE), static_cast<unsigned>(rows < 65535 ? rows : 65535)), 256, 0, c.stream>>>(p);
    return cudaGetLastError();
}

// ws: 2 n f fp32, then (nothing to keep) 3 n f of T
template <typename T> int forward(const Call &c, T *y, T *kept, float *ws) {
    const int64_t nf = c.n * c.f;
    if (kept == nullptr) kept = reinterpret_cast<T *>(ws + 2 * nf);
    T *m = kept + 2 * nf;
    const T *W = static_cast<const T *>(c.W_in);
    cudaError_t e = product<T>(c, c.x, c.d, 1, W, c.d, 1, c.n, c.f, c.d, ws, c.f);
    if (e == cudaSuccess) e = product<T>(c, c.x, c.d, 1, W + c.f * c.d, c.d, 1, c.n, c.f, c.d, ws + nf, c.f);
    if (e != cudaSuccess) return NRNN_ERR_CUDA;
    k_gate<T><<<1024, 256, 0, c.stream>>>(ws, ws + nf, kept, kept + nf, m, nf);
    e = product<T>(c, m, c.f, 1, c.W_out, c.f, 1, c.n, c.d, c.f, y, c.d);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

// ws: n f fp32 of gm, 2 n f of T, n d fp32 of gx
template <typename T>
int backward(const Call &c, const T *kept, const void *g, T *gx, T *gW_in, T *gW_out, float *ws) {
    const int64_t nf = c.n * c.f;
    const T *a = kept, *b = a + nf, *m = b + nf;
    float *gm = ws, *sum = gm + nf;
    T *ga = reinterpret_cast<T *>(sum + c.n * c.d), *gb = ga + nf;
    const T *W = static_cast<const T *>(c.W_in);
    cudaError_t e = product<T>(c, g, c.d, 1, c.W_out, 1, c.f, c.n, c.f, c.d, gm, c.f);
    if (e != cudaSuccess) return NRNN_ERR_CUDA;
    k_gate_back<T><<<1024, 256, 0, c.stream>>>(a, b, gm, ga, gb, nf);
    e = product<T>(c, ga, c.f, 1, W, 1, c.d, c.n, c.d, c.f, sum, c.d);
    if (e == cudaSuccess) e = product<T>(c, gb, c.f, 1, W + c.f * c.d, 1, c.d, c.n, c.d, c.f, sum, c.d, true);
    if (e == cudaSuccess) e = product<T>(c, ga, 1, c.f, c.x, 1, c.d, c.f, c.d, c.n, gW_in, c.d);
    if (e == cudaSuccess) e = product<T>(c, gb, 1, c.f, c.x, 1, c.d, c.f, c.d, c.n, gW_in + c.f * c.d, c.d);
    if (e == cudaSuccess) e = product<T>(c, g, 1, c.d, m, 1, c.f, c.d, c.f, c.n, gW_out, c.f);
    if (e != cudaSuccess) return NRNN_ERR_CUDA;
    k_round<T><<<1024, 256, 0, c.stream>>>(sum, gx, c.n * c.d);
    return cudaGetLastError() == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

bool sizes_fit(int64_t n, int64_t d, int64_t f) { return n <= (1 << 30) && d <= (1 << 20) && f <= (1 << 20); }

int check(const Call &c) {
    if (c.dtype != NRNN_F32 && c.dtype != NRNN_BF16) return NRNN_ERR_INVALID_ARG;
    if (c.n < 0 || c.d <= 0 || c.f <= 0) return NRNN_ERR_INVALID_ARG;
    if (!sizes_fit(c.n, c.d, c.f)) return NRNN_ERR_UNSUPPORTED;
    const uintptr_t elem = c.dtype == NRNN_BF16 ? 2 : 4;
    if (c.W_in == nullptr || c.W_out == nullptr || (c.n > 0 && c.x == nullptr)) return NRNN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(c.x) | reinterpret_cast<uintptr_t>(c.W_in) | reinterpret_cast<uintptr_t>(c.W_out)) % elem != 0)
        return NRNN_ERR_INVALID_ARG;
    return NRNN_OK;
}

bool usable(const void *ws, size_t have, size_t need) {
    return ws != nullptr && reinterpret_cast<uintptr_t>(ws) % 256 == 0 && have >= need;
}

}  // namespace
}  // namespace nrnn

using namespace nrnn;

extern "C" {

size_t nrnn_gated_mlp_kept_bytes(int64_t rows, int64_t f, int dtype) {
    if (rows < 0 || f <= 0 || !sizes_fit(rows, 1, f) || (dtype != NRNN_F32 && dtype != NRNN_BF16)) return 0;
    return up256(3 * (dtype == NRNN_BF16 ? 2 : 4) * rows * f + 1);
}

size_t nrnn_gated_mlp_workspace_bytes(int64_t rows, int64_t d, int64_t f, int dtype, int backward) {
    if (d <= 0 || !sizes_fit(0, d, 1) || nrnn_gated_mlp_kept_bytes(rows, f, dtype) == 0) return 0;
    const size_t elem = dtype == NRNN_BF16 ? 2 : 4;
    return up256(rows * f * (backward ? 4 + 2 * elem : 8 + 3 * elem) + (backward ? 4 * rows * d : 0) + 1);
}

int nrnn_gated_mlp_forward(const void *x, const void *W_in, const void *W_out, int dtype, int64_t rows, int64_t d,
                           int64_t f, void *y, void *kept, void *workspace, size_t ws_bytes, void *stream) {
    const Call c{x, W_in, W_out, dtype, rows, d, f, static_cast<cudaStream_t>(stream)};
    const int st = check(c);
    if (st != NRNN_OK) return st;
    if (rows == 0) return NRNN_OK;
    const uintptr_t elem = dtype == NRNN_BF16 ? 2 : 4;
    if (y == nullptr || reinterpret_cast<uintptr_t>(y) % elem != 0 || reinterpret_cast<uintptr_t>(kept) % 256 != 0)
        return NRNN_ERR_INVALID_ARG;
    if (!usable(workspace, ws_bytes, nrnn_gated_mlp_workspace_bytes(rows, d, f, dtype, 0))) return NRNN_ERR_WORKSPACE;
    float *ws = static_cast<float *>(workspace);
    return dtype == NRNN_BF16 ? forward(c, static_cast<__nv_bfloat16 *>(y), static_cast<__nv_bfloat16 *>(kept), ws)
                              : forward(c, static_cast<float *>(y), static_cast<float *>(kept), ws);
}

int nrnn_gated_mlp_backward(const void *x, const void *W_in, const void *W_out, const void *kept, const void *g,
                            int dtype, int64_t rows, int64_t d, int64_t f, void *gx, void *gW_in, void *gW_out,
                            void *workspace, size_t ws_bytes, void *stream) {
    const Call c{x, W_in, W_out, dtype, rows, d, f, static_cast<cudaStream_t>(stream)};
    const int st = check(c);
    if (st != NRNN_OK) return st;
    const uintptr_t elem = dtype == NRNN_BF16 ? 2 : 4;
    if (gW_in == nullptr || gW_out == nullptr ||
        (rows > 0 && (g == nullptr || gx == nullptr || kept == nullptr || reinterpret_cast<uintptr_t>(kept) % 256 != 0)) ||
        (reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(gx) | reinterpret_cast<uintptr_t>(gW_in) |
         reinterpret_cast<uintptr_t>(gW_out)) % elem != 0)
        return NRNN_ERR_INVALID_ARG;
    if (rows == 0)
        return cudaMemsetAsync(gW_in, 0, elem * 2 * f * d, c.stream) == cudaSuccess &&
                       cudaMemsetAsync(gW_out, 0, elem * f * d, c.stream) == cudaSuccess
                   ? NRNN_OK : NRNN_ERR_CUDA;
    if (!usable(workspace, ws_bytes, nrnn_gated_mlp_workspace_bytes(rows, d, f, dtype, 1))) return NRNN_ERR_WORKSPACE;
    return dtype == NRNN_BF16
               ? backward<__nv_bfloat16>(c, static_cast<const __nv_bfloat16 *>(kept), g, static_cast<__nv_bfloat16 *>(gx),
                                         static_cast<__nv_bfloat16 *>(gW_in), static_cast<__nv_bfloat16 *>(gW_out),
                                         static_cast<float *>(workspace))
               : backward<float>(c, static_cast<const float *>(kept), g, static_cast<float *>(gx), static_cast<float *>(gW_in),
                                 static_cast<float *>(gW_out), static_cast<float *>(workspace));
}

}  // extern "C"
