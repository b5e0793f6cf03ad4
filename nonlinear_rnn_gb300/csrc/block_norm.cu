// The norms before and after a block, fused with the block's gate and the
// residual scale.
//
//   n  = h rsqrt(mean(h^2) + eps)          the block's output, normalised
//   y  = n w_post silu(gate)               (no gate: y = n w_post)
//   x' = x + scale y                       the residual stream
//   u  = x' rsqrt(mean(x'^2) + eps) w_pre  the next block's input
//
// Backward, from the stored x', h and gate and the gradients gx' and gu (a hat
// is a normalised row, r and q the two reciprocal roots, <.> a row's mean):
//
//   t    = gx' + r (a - x^ <a x^>),  a = gu w_pre       = dL/dx, and dL/d(scale y)
//   gh   = q (b - h^ <b h^>),        b = t scale silu(gate) w_post
//   ggate = t scale h^ w_post silu'(gate)
//   gw_pre = sum gu x^,  gscale = sum t y,  gw_post = sum t scale silu(gate) h^
//
// Neither direction has a product to speak of: both are bound by HBM, 5 row
// passes forward (x, h, gate in; x', u out) and 8 backward (x', h, gate, gx',
// gu in; gx, gh, ggate out).  A row is read once and stays in registers; the
// statistics are recomputed in the backward from the row it reads anyway
// instead of being stored.  All arithmetic and all sums are fp32.
#include "../../include/nrnn.h"
#include "nrnn_device.cuh"
#include "nrnn_internal.h"
#include "rows.cuh"

namespace nrnn {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int MAX_D = 8192;   // a row in the registers of one CTA

__device__ __forceinline__ float sigmoid(float v) {
    return __fdividef(1.f, 1.f + ex2_approx(-v * LOG2E));
}

template <int TPR> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}

struct NormArgs {
    const void *x, *h, *gate;            // x: x' in the backward
    const float *w_post, *scale, *w_pre; // null: ones
    const void *g_x, *g_u;               // backward: null = zeros
    void *out_x, *out_u;                 // forward: x', u
    void *gx, *gh, *g_gate;
    float *part;                         // backward: [CTAs][3][d] sums of the weights' gradients
    int64_t rows;
    int d;
    float eps;
    bool norm_u;                         // u is wanted (forward), w_pre's branch exists (backward)
};

// E columns of a row per thread, as E / VEC vectors TPR vectors apart
template <typename T, int VEC, int E>
__device__ __forceinline__ void load_row(const void *base, int64_t row, int d, int c0, int step,
                                         float (&f)[E]) {
    const T *p = static_cast<const T *>(base) + row * d;
#pragma unroll
    for (int i = 0; i < E / VEC; ++i) {
        const int c = c0 + i * step;
        float v[VEC] = {};
        if (c < d) load_f32<T, VEC>(p + c, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[i * VEC + e] = v[e];
    }
}
template <typename T, int VEC, int E>
__device__ __forceinline__ void store_row(void *base, int64_t row, int d, int c0, int step,
                                          const float (&f)[E]) {
    T *p = static_cast<T *>(base) + row * d;
#pragma unroll
    for (int i = 0; i < E / VEC; ++i) {
        const int c = c0 + i * step;
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = f[i * VEC + e];
        if (c < d) store_f32<T, VEC>(p + c, v);
    }
}
// the threads' E columns of a (d) fp32 vector; null = ones
template <int VEC, int E>
__device__ __forceinline__ void load_weight(const float *w, int d, int c0, int step, float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E / VEC; ++i) {
        const int c = c0 + i * step;
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[i * VEC + e] = w == nullptr ? 1.f : c < d ? __ldg(w + c + e) : 0.f;
    }
}

// ------------------------------------------------------------------- forward
// TPR threads a row (a power of two up to a warp), or a whole CTA (TPR = 256)
// for rows of more than 32 E columns.
constexpr int FWD_THREADS = 256;

template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *smem) {
    if (TPR <= 32) return lanes_sum<TPR>(v);
    v = lanes_sum<32>(v);
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) s += smem[w];
    return s;
}

template <typename T, int VEC, int E, int TPR>
__global__ void __launch_bounds__(FWD_THREADS) k_norm_forward(const NormArgs a) {
    __shared__ float red[2][FWD_THREADS / 32];
    const int t = threadIdx.x % TPR;
    const int64_t row = blockIdx.x * static_cast<int64_t>(FWD_THREADS / TPR) + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const int64_t at = live ? row : a.rows - 1;   // threads past the end repeat the last row unstored
    const int c0 = t * VEC, step = TPR * VEC;
    float x[E], v[E], w[E];
    load_row<T, VEC>(a.x, at, a.d, c0, step, x);
    if (a.h != nullptr) {
        load_row<T, VEC>(a.h, at, a.d, c0, step, v);
        float gate[E];
        if (a.gate != nullptr) load_row<T, VEC>(a.gate, at, a.d, c0, step, gate);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(v[e], v[e], ss);
        const float q = rsqrtf(row_sum<TPR>(ss, red[0]) / a.d + a.eps);
        load_weight<VEC>(a.w_post, a.d, c0, step, w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= q * w[e];
        if (a.gate != nullptr) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= gate[e] * sigmoid(gate[e]);
        }
        load_weight<VEC>(a.scale, a.d, c0, step, w);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fmaf(w[e], v[e], x[e]);
        if (live) store_row<T, VEC>(a.out_x, row, a.d, c0, step, x);
    }
    if (!a.norm_u) return;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < E / VEC; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (c0 + i * step < a.d) ss = fmaf(x[i * VEC + e], x[i * VEC + e], ss);
    const float r = rsqrtf(row_sum<TPR>(ss, red[1]) / a.d + a.eps);
    load_weight<VEC>(a.w_pre, a.d, c0, step, w);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= r * w[e];
    if (live) store_row<T, VEC>(a.out_u, row, a.d, c0, step, x);
}

// ------------------------------------------------------------------ backward
// Persistent CTAs; blockDim.x <= TPR threads a row, or (TPR = 32) a warp a row
// and BWD_WARPS rows a CTA.  Each thread keeps its E columns of the
// weights and of their gradients in registers over all its rows.
constexpr int BWD_E = 8, BWD_WARPS = 4;

// sums of N values over a row's threads; buf: [2][N][32], used in turn
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *buf) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<32>(v[i]);
    if (TPR == 32) return;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i * 32 + (threadIdx.x >> 5)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += buf[i * 32 + w];
        v[i] = s;
    }
}

template <typename T, int VEC, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? BWD_WARPS * 32 : TPR) k_norm_backward(const NormArgs a) {
    constexpr int E = BWD_E;
    __shared__ float red[2][4 * 32];   // three sums, then one; two rows in turn
    extern __shared__ float join[];    // TPR = 32: [3][d]
    const int tpr = TPR == 32 ? 32 : blockDim.x;
    const int t = threadIdx.x % tpr, group = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const int c0 = t * VEC, step = tpr * VEC;
    const float inv_d = 1.f / a.d;
    float w_post[E], scale[E], w_pre[E];
    load_weight<VEC>(a.w_post, a.d, c0, step, w_post);
    load_weight<VEC>(a.scale, a.d, c0, step, scale);
    load_weight<VEC>(a.w_pre, a.d, c0, step, w_pre);
    float s_post[E] = {}, s_scale[E] = {}, s_pre[E] = {};
    int turn = 0;
    for (int64_t row = blockIdx.x * static_cast<int64_t>(groups) + group; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * groups, turn ^= 1) {
        float x[E] = {}, h[E] = {}, gate[E], gx[E] = {}, gu[E] = {};
        if (a.norm_u) {
            load_row<T, VEC>(a.x, row, a.d, c0, step, x);
            load_row<T, VEC>(a.g_u, row, a.d, c0, step, gu);
        }
        if (a.g_x != nullptr) load_row<T, VEC>(a.g_x, row, a.d, c0, step, gx);
        if (a.h != nullptr) load_row<T, VEC>(a.h, row, a.d, c0, step, h);
        if (a.gate != nullptr) load_row<T, VEC>(a.gate, row, a.d, c0, step, gate);
        float m[3] = {};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            m[0] = fmaf(x[e], x[e], m[0]);
            m[1] = fmaf(gu[e] * w_pre[e], x[e], m[1]);
            m[2] = fmaf(h[e], h[e], m[2]);
        }
        row_sums<TPR, 3>(m, red[turn]);
        const float r = rsqrtf(m[0] * inv_d + a.eps), q = rsqrtf(m[2] * inv_d + a.eps);
        const float mean_ax = m[1] * inv_d * r;   // <a x^>
        if (a.norm_u) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float xn = x[e] * r;
                s_pre[e] = fmaf(gu[e], xn, s_pre[e]);
                gx[e] = fmaf(r, fmaf(-xn, mean_ax, gu[e] * w_pre[e]), gx[e]);   // t
            }
        }
        store_row<T, VEC>(a.gx, row, a.d, c0, step, gx);
        if (a.h == nullptr) continue;
        float k[1] = {};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float hn = h[e] * q;
            float of = 1.f, slope = 0.f;
            if (a.gate != nullptr) {
                const float s = sigmoid(gate[e]);
                of = gate[e] * s;
                slope = s * fmaf(gate[e], 1.f - s, 1.f);
            }
            const float n = hn * w_post[e], gy = gx[e] * scale[e];
            s_scale[e] = fmaf(gx[e], n * of, s_scale[e]);
            s_post[e] = fmaf(gy * of, hn, s_post[e]);
            gate[e] = gy * n * slope;      // dL/dgate
            gx[e] = gy * of * w_post[e];   // b
            h[e] = hn;
            k[0] = fmaf(gx[e], hn, k[0]);
        }
        if (a.gate != nullptr) store_row<T, VEC>(a.g_gate, row, a.d, c0, step, gate);
        row_sums<TPR, 1>(k, red[turn] + 3 * 32);
        const float mean_bh = k[0] * inv_d;
#pragma unroll
        for (int e = 0; e < E; ++e) gx[e] = q * fmaf(-h[e], mean_bh, gx[e]);
        store_row<T, VEC>(a.gh, row, a.d, c0, step, gx);
    }
    // this CTA's sums: warps of a CTA in order (TPR = 32), then to the workspace
    float *part = a.part + blockIdx.x * static_cast<int64_t>(3) * a.d;
    for (int g = 0; g < groups; ++g) {
        if (TPR == 32) __syncthreads();
        if (g != group) continue;
        float *to = TPR == 32 && g < groups - 1 ? join : part;
#pragma unroll
        for (int i = 0; i < E / VEC; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = c0 + i * step + e, o = i * VEC + e;
                if (c >= a.d) continue;
                float v[3] = {s_post[o], s_scale[o], s_pre[o]};
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    if (TPR == 32 && g > 0) v[q] += join[q * a.d + c];
                    to[q * a.d + c] = v[q];
                }
            }
    }
}

// sums of the CTAs' partial sums, in order: a warp's lanes take 32 columns, the
// warps of the CTA every JOIN_WARPS-th partial
constexpr int JOIN_WARPS = 16;

__global__ void __launch_bounds__(JOIN_WARPS * 32)
    k_norm_join(const float *__restrict__ part, int n_part, int d, float *gw_post, float *g_scale,
                float *gw_pre) {
    __shared__ float sum[JOIN_WARPS][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;   // column of [3][d]
    float s = 0.f;
    if (c < 3 * d) {
#pragma unroll 4
        for (int p = w; p < n_part; p += JOIN_WARPS) s += part[static_cast<int64_t>(p) * 3 * d + c];
    }
    sum[w][lane] = s;
    __syncthreads();
    if (w > 0 || c >= 3 * d) return;
#pragma unroll
    for (int q = 1; q < JOIN_WARPS; ++q) s += sum[q][lane];
    float *to = c < d ? gw_post : c < 2 * d ? g_scale : gw_pre;
    if (to != nullptr) to[c % d] = s;
}

// ---------------------------------------------------------------- host side
bool aligned_to(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename T, int VEC, int E, int TPR>
cudaError_t forward_as(const NormArgs &a, cudaStream_t s) {
    const int64_t blocks = (a.rows + FWD_THREADS / TPR - 1) / (FWD_THREADS / TPR);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    k_norm_forward<T, VEC, E, TPR><<<static_cast<unsigned>(blocks), FWD_THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

// the fewest threads a row that hold it in at most 32 columns each
template <typename T, int VEC> cudaError_t forward_for(const NormArgs &a, cudaStream_t s) {
    constexpr int E = 32;
    if (a.d <= 8 * 8) return forward_as<T, VEC, 8, 8>(a, s);
    if (a.d <= 8 * E) return forward_as<T, VEC, E, 8>(a, s);
    if (a.d <= 16 * E) return forward_as<T, VEC, E, 16>(a, s);
    if (a.d <= 32 * E) return forward_as<T, VEC, E, 32>(a, s);
    return forward_as<T, VEC, E, 256>(a, s);
}

// 608 = 152 SMs x 4: the CTAs of a backward launch for long inputs
constexpr int BWD_CTAS = 608;

int backward_ctas(int64_t rows, int d) {
    const int64_t per = d <= 32 * BWD_E ? BWD_WARPS : 1;
    const int64_t want = (rows + per - 1) / per;
    return static_cast<int>(want < BWD_CTAS ? want : BWD_CTAS);
}

template <typename T, int VEC> cudaError_t backward_for(const NormArgs &a, int ctas, cudaStream_t s) {
    if (a.d <= 32 * BWD_E) {
        k_norm_backward<T, VEC, 32><<<ctas, BWD_WARPS * 32, sizeof(float) * 3 * a.d, s>>>(a);
    } else {
        const int threads = ((a.d + BWD_E - 1) / BWD_E + 31) / 32 * 32;
        if (threads <= 128) k_norm_backward<T, VEC, 128><<<ctas, threads, 0, s>>>(a);
        else k_norm_backward<T, VEC, 1024><<<ctas, threads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

int check_norm(int dtype, int64_t rows, int64_t d, float eps) {
    if (dtype != NRNN_F32 && dtype != NRNN_BF16) return NRNN_ERR_INVALID_ARG;
    if (rows < 0 || d <= 0 || !(eps >= 0.f)) return NRNN_ERR_INVALID_ARG;
    if (d > MAX_D) return NRNN_ERR_UNSUPPORTED;
    return NRNN_OK;
}

// widest access of 16 bytes, or one element
int width_for(int elem, int64_t d, std::initializer_list<const void *> ptrs) {
    const int vec = 16 / elem;
    if (d % vec != 0) return 1;
    for (const void *p : ptrs)
        if (!aligned_to(p, 16)) return 1;
    return vec;
}

}  // namespace
}  // namespace nrnn

using namespace nrnn;

extern "C" {

int nrnn_block_norm_forward(const void *x, const void *h, const void *gate, const float *w_post,
                            const float *scale, const float *w_pre, int dtype, int64_t rows,
                            int64_t d, float eps, void *x_out, void *u, void *stream) {
    const int st = check_norm(dtype, rows, d, eps);
    if (st != NRNN_OK) return st;
    if (rows == 0) return NRNN_OK;
    if (h == nullptr && (gate != nullptr || u == nullptr)) return NRNN_ERR_INVALID_ARG;
    if (x == nullptr || (h != nullptr && x_out == nullptr)) return NRNN_ERR_INVALID_ARG;
    const int elem = dtype == NRNN_BF16 ? 2 : 4;
    for (const void *p : {x, h, gate, static_cast<const void *>(x_out), static_cast<const void *>(u)})
        if (!aligned_to(p, elem)) return NRNN_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = x; a.h = h; a.gate = gate;
    a.w_post = w_post; a.scale = scale; a.w_pre = w_pre;
    a.out_x = x_out; a.out_u = u;
    a.rows = rows; a.d = static_cast<int>(d); a.eps = eps;
    a.norm_u = u != nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool wide = width_for(elem, d, {x, h, gate, x_out, u}) > 1;
    cudaError_t e;
    if (dtype == NRNN_BF16)
        e = wide ? forward_for<__nv_bfloat16, 8>(a, s) : forward_for<__nv_bfloat16, 1>(a, s);
    else
        e = wide ? forward_for<float, 4>(a, s) : forward_for<float, 1>(a, s);
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

size_t nrnn_block_norm_backward_workspace_bytes(int64_t rows, int64_t d) {
    if (rows < 0 || d <= 0 || d > MAX_D) return 0;
    const size_t bytes = sizeof(float) * 3 * d * (rows > 0 ? backward_ctas(rows, static_cast<int>(d)) : 1);
    return (bytes + 255) / 256 * 256;
}

int nrnn_block_norm_backward(const void *x_out, const void *h, const void *gate,
                             const float *w_post, const float *scale, const float *w_pre,
                             const void *g_x, const void *g_u, int dtype, int64_t rows, int64_t d,
                             float eps, void *gx, void *gh, void *g_gate, float *gw_post,
                             float *g_scale, float *gw_pre, void *workspace, size_t ws_bytes,
                             void *stream) {
    const int st = check_norm(dtype, rows, d, eps);
    if (st != NRNN_OK) return st;
    if (rows > 0) {
        if (g_x == nullptr && g_u == nullptr) return NRNN_ERR_INVALID_ARG;
        if (h == nullptr && (gate != nullptr || g_u == nullptr)) return NRNN_ERR_INVALID_ARG;
        if (gx == nullptr || (g_u != nullptr && x_out == nullptr) || (h != nullptr && gh == nullptr) ||
            (gate != nullptr && g_gate == nullptr))
            return NRNN_ERR_INVALID_ARG;
    }
    const int elem = dtype == NRNN_BF16 ? 2 : 4;
    for (const void *p : {x_out, h, gate, g_x, g_u, static_cast<const void *>(gx),
                          static_cast<const void *>(gh), static_cast<const void *>(g_gate)})
        if (!aligned_to(p, elem)) return NRNN_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned_to(workspace, 256) ||
        ws_bytes < nrnn_block_norm_backward_workspace_bytes(rows, d))
        return NRNN_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    NormArgs a{};
    a.x = x_out; a.h = h; a.gate = gate;
    a.w_post = w_post; a.scale = scale; a.w_pre = w_pre;
    a.g_x = g_x; a.g_u = g_u;
    a.gx = gx; a.gh = gh; a.g_gate = g_gate;
    a.part = static_cast<float *>(workspace);
    a.rows = rows; a.d = static_cast<int>(d); a.eps = eps;
    a.norm_u = g_u != nullptr;
    const int ctas = rows > 0 ? backward_ctas(rows, a.d) : 0;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        const bool wide = width_for(elem, d, {x_out, h, gate, g_x, g_u, gx, gh, g_gate}) > 1;
        if (dtype == NRNN_BF16)
            e = wide ? backward_for<__nv_bfloat16, 8>(a, ctas, s) : backward_for<__nv_bfloat16, 1>(a, ctas, s);
        else
            e = wide ? backward_for<float, 4>(a, ctas, s) : backward_for<float, 1>(a, ctas, s);
    }
    if (e == cudaSuccess) {
        k_norm_join<<<(3 * a.d + 31) / 32, JOIN_WARPS * 32, 0, s>>>(a.part, ctas, a.d, gw_post, g_scale,
                                                                   gw_pre);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

}  // extern "C"
