// Gated linear recurrence: a diagonal recurrence whose gates do not depend on the
// state, so that it needs one scan and no Newton iterations.
//
//   r = sig(P_a + b_a),  a = exp(-rate r),  i = sig(P_i + b_i),  s = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + s_t i_t v_t,   preactivation blocks [a | i | v]
//
// s keeps the state's variance that of i v whatever the decay.  Its gradient, at the
// states as stored, with G_t = gH_t + a_{t+1} G_{t+1}:
//
//   w = G (a h_{t-1} - (a^2 / s) i v)                       (dL/d log a)
//   gP_a = -w rate r (1 - r),  g_rate = -sum w r,  g_b_a = sum gP_a
//   gP_i = G s v i (1 - i),    g_b_i = sum gP_i,   gP_v = G s i
//
// r and i are bounded below by 2^-63 (the exponential is clamped, so that 1 - r is
// exact to rounding on both sides); where s is zero all the same (a rate of zero)
// the term with a^2 / s is left out, which is its limit as r vanishes.
#include "../../include/nrnn.h"
#include "nrnn_device.cuh"
#include "nrnn_internal.h"

namespace nrnn {
namespace {

struct Gates {
    float a, s;        // decay, sqrt(1 - a^2)
    float r, omr;      // r, 1 - r
    float i, omi;
};

__device__ __forceinline__ void sigmoid_both(float x, float &s, float &oms) {
    const float e = ex2_approx(min_nan(-LOG2E * x, EXP2_CLAMP));
    s = rcp_approx(1.0f + e);
    oms = e * s;
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 - e^-y: below 1/4 by its series to y^6 / 720, where the difference would lose bits
__device__ __forceinline__ float one_less_exp(float y, float e) {
    const float p = y * fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 720, 1.f / 120), -1.f / 24), 1.f / 6), -0.5f), 1.f);
    return y < 0.25f ? p : 1.f - e;
}

__device__ __forceinline__ Gates gates_of(float pa, float pi, float rate, float b_a, float b_i) {
    Gates g;
    sigmoid_both(pa + b_a, g.r, g.omr);
    sigmoid_both(pi + b_i, g.i, g.omi);
    const float fall = rate * g.r;
    g.a = ex2_approx(-LOG2E * fall);
    g.s = sqrt_approx(one_less_exp(2.f * fall, g.a * g.a));
    return g;
}

constexpr int SEQ_THREADS = 128;

struct RecArgs {
    const void *P, *H, *gH;
    const float *params, *state;      // state (rows, d) or null
    const int32_t *cu;
    int rows;                         // sequences: B or segments
    int64_t T;
    int d;
    void *H_out;
    float *last;                      // (rows, d) or null
    const float *g_last;
    void *gP;
    float *g_state, *gparams;
    float *part;                      // (rows, 3, d) sums of the parameters' gradients
};

__device__ __forceinline__ void span_of(const RecArgs &a, int row, int64_t &t0, int64_t &t1) {
    if (a.cu == nullptr) {
        t0 = row * a.T;
        t1 = t0 + a.T;
        return;
    }
    t0 = min(max(static_cast<int64_t>(__ldg(a.cu + row)), static_cast<int64_t>(0)), a.T);
    t1 = min(max(static_cast<int64_t>(__ldg(a.cu + row + 1)), t0), a.T);
}

template <typename TS>
__global__ void __launch_bounds__(SEQ_THREADS) k_forward(const RecArgs a) {
    const int u = blockIdx.x * SEQ_THREADS + threadIdx.x;
    if (u >= a.d) return;
    const float rate = a.params[u], b_a = a.params[a.d + u], b_i = a.params[2 * a.d + u];
    for (int row = blockIdx.y; row < a.rows; row += gridDim.y) {
        int64_t t0, t1;
        span_of(a, row, t0, t1);
        const int64_t at = static_cast<int64_t>(row) * a.d + u;
        float h = a.state != nullptr ? a.state[at] : 0.f;
        for (int64_t t = t0; t < t1; ++t) {
            const TS *p = static_cast<const TS *>(a.P) + t * 3 * a.d + u;
            const Gates g = gates_of(to_f32(p[0]), to_f32(p[a.d]), rate, b_a, b_i);
            h = fmaf(g.a, h, g.s * g.i * to_f32(p[2 * a.d]));
            static_cast<TS *>(a.H_out)[t * a.d + u] = from_f32<TS>(h);
        }
        if (a.last != nullptr) a.last[at] = h;
    }
}

template <typename TS>
__global__ void __launch_bounds__(SEQ_THREADS) k_backward(const RecArgs a) {
    const int u = blockIdx.x * SEQ_THREADS + threadIdx.x;
    if (u >= a.d) return;
    const float rate = a.params[u], b_a = a.params[a.d + u], b_i = a.params[2 * a.d + u];
    for (int row = blockIdx.y; row < a.rows; row += gridDim.y) {
        int64_t t0, t1;
        span_of(a, row, t0, t1);
        const int64_t at = static_cast<int64_t>(row) * a.d + u;
        float nu = a.g_last != nullptr ? a.g_last[at] : 0.f;
        float g_rate = 0.f, g_ba = 0.f, g_bi = 0.f;
        for (int64_t t = t1 - 1; t >= t0; --t) {
            const TS *p = static_cast<const TS *>(a.P) + t * 3 * a.d + u;
            const Gates g = gates_of(to_f32(p[0]), to_f32(p[a.d]), rate, b_a, b_i);
            const float v = to_f32(p[2 * a.d]);
            const float before = t > t0 ? to_f32(static_cast<const TS *>(a.H)[(t - 1) * a.d + u])
                                        : a.state != nullptr ? a.state[at] : 0.f;
            const float G = to_f32(static_cast<const TS *>(a.gH)[t * a.d + u]) + nu;
            nu = g.a * G;
            const float over = g.s > 0.f ? g.a * rcp_approx(g.s) : 0.f;
            const float w = nu * (before - over * g.i * v);
            const float wr = w * g.r;
            const float ga = -rate * wr * g.omr, gv = G * g.s * g.i, gi = gv * v * g.omi;
            TS *o = static_cast<TS *>(a.gP) + t * 3 * a.d + u;
            o[0] = from_f32<TS>(ga);
            o[a.d] = from_f32<TS>(gi);
            o[2 * a.d] = from_f32<TS>(gv);
            g_rate -= wr;
            g_ba += ga;
            g_bi += gi;
        }
        if (a.g_state != nullptr) a.g_state[at] = nu;
        float *part = a.part + static_cast<int64_t>(row) * 3 * a.d + u;
        part[0] = g_rate;
        part[a.d] = g_ba;
        part[2 * a.d] = g_bi;
    }
}

// sums of the parameters' gradients over the rows, in order
__global__ void __launch_bounds__(128) k_join(const float *part, int rows, int n, float *out) {
    const int j = blockIdx.x * 128 + threadIdx.x;
    if (j >= n) return;
    float s = 0.f;
    for (int r = 0; r < rows; ++r) s += part[static_cast<int64_t>(r) * n + j];
    out[j] = s;
}

template <typename TS>
__global__ void __launch_bounds__(256)
    k_step(const TS *P, const float *params, const float *state, int64_t n, int d, TS *h_out, float *last) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t slot = i / d;
    const int u = static_cast<int>(i - slot * d);
    const TS *p = P + slot * 3 * d + u;
    const Gates g = gates_of(to_f32(p[0]), to_f32(p[d]), params[u], params[d + u], params[2 * d + u]);
    const float h = fmaf(g.a, state != nullptr ? state[i] : 0.f, g.s * g.i * to_f32(p[2 * d]));
    h_out[i] = from_f32<TS>(h);
    last[i] = h;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check(const void *P, int dtype, const float *params, int64_t B, int64_t T, int64_t d,
          const int32_t *cu, int64_t S) {
    if (dtype != NRNN_F32 && dtype != NRNN_BF16) return NRNN_ERR_INVALID_ARG;
    if (B < 0 || T < 0 || d <= 0 || S < 0) return NRNN_ERR_INVALID_ARG;
    if (B > INT32_MAX || T > INT32_MAX || d > (1 << 24) || S > INT32_MAX - 1 || d % 8 != 0)
        return NRNN_ERR_UNSUPPORTED;
    if (B > 0 && T > (INT64_MAX >> 8) / (B * d)) return NRNN_ERR_UNSUPPORTED;
    if (cu != nullptr && (B != 1 || S < 1)) return NRNN_ERR_CU_SEQLENS;
    if (params == nullptr || !aligned16(params)) return NRNN_ERR_INVALID_ARG;
    if (B * T > 0 && (P == nullptr || !aligned16(P))) return NRNN_ERR_INVALID_ARG;
    return NRNN_OK;
}

bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    if (a == nullptr || b == nullptr) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

}  // namespace
}  // namespace nrnn

using namespace nrnn;

extern "C" {

size_t nrnn_linear_recurrence_workspace_bytes(int64_t B, int64_t T, int64_t d_h, int dtype,
                                              int64_t num_segments, int backward) {
    if (B < 0 || T < 0 || d_h <= 0 || d_h > (1 << 24) || num_segments < 0 ||
        (dtype != NRNN_F32 && dtype != NRNN_BF16))
        return 0;
    const int64_t rows = num_segments > 0 ? num_segments : B;
    return 256 + (backward ? sizeof(float) * 3 * d_h * rows : 0);
}

int nrnn_linear_recurrence_forward(const void *preact, int dtype, const float *params, int64_t B,
                                   int64_t T, int64_t d_h, const int32_t *cu_seqlens,
                                   int64_t num_segments, const float *state, void *H, float *last,
                                   void *workspace, size_t ws_bytes, void *stream) {
    const int st = check(preact, dtype, params, B, T, d_h, cu_seqlens, num_segments);
    if (st != NRNN_OK) return st;
    const int64_t es = dtype == NRNN_BF16 ? 2 : 4, n = B * T * d_h;
    const int64_t rows = cu_seqlens != nullptr ? num_segments : B;
    if ((n > 0 && (H == nullptr || !aligned16(H))) || !aligned16(state) || !aligned16(last) ||
        overlap(preact, 3 * n * es, H, n * es) || overlap(state, rows * d_h * 4, H, n * es) ||
        (state != last && overlap(state, rows * d_h * 4, last, rows * d_h * 4)))
        return NRNN_ERR_INVALID_ARG;
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
        ws_bytes < nrnn_linear_recurrence_workspace_bytes(B, T, d_h, dtype, cu_seqlens ? num_segments : 0, 0))
        return NRNN_ERR_WORKSPACE;
    if (rows == 0) return NRNN_OK;
    RecArgs a{};
    a.P = preact; a.params = params; a.state = state; a.cu = cu_seqlens;
    a.rows = static_cast<int>(rows); a.T = T; a.d = static_cast<int>(d_h);
    a.H_out = H; a.last = last;
    const dim3 grid(static_cast<unsigned>((d_h + SEQ_THREADS - 1) / SEQ_THREADS), static_cast<unsigned>(rows < 65535 ? rows : 65535));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == NRNN_BF16) k_forward<__nv_bfloat16><<<grid, SEQ_THREADS, 0, s>>>(a);
    else k_forward<float><<<grid, SEQ_THREADS, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

int nrnn_linear_recurrence_backward(const void *preact, int dtype, const float *params, int64_t B,
                                    int64_t T, int64_t d_h, const int32_t *cu_seqlens,
                                    int64_t num_segments, const float *state, const void *H,
                                    const void *gH, const float *g_last, void *gP, float *gparams,
                                    float *g_state, void *workspace, size_t ws_bytes, void *stream) {
    const int st = check(preact, dtype, params, B, T, d_h, cu_seqlens, num_segments);
    if (st != NRNN_OK) return st;
    const int64_t es = dtype == NRNN_BF16 ? 2 : 4, n = B * T * d_h;
    const int64_t rows = cu_seqlens != nullptr ? num_segments : B;
    if (gparams == nullptr || !aligned16(gparams) || !aligned16(state) || !aligned16(g_last) || !aligned16(g_state) ||
        (n > 0 && (H == nullptr || gH == nullptr || gP == nullptr || !aligned16(H) || !aligned16(gH) || !aligned16(gP))) ||
        overlap(preact, 3 * n * es, gP, 3 * n * es) || overlap(H, n * es, gP, 3 * n * es) ||
        overlap(gH, n * es, gP, 3 * n * es))
        return NRNN_ERR_INVALID_ARG;
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
        ws_bytes < nrnn_linear_recurrence_workspace_bytes(B, T, d_h, dtype, cu_seqlens ? num_segments : 0, 1))
        return NRNN_ERR_WORKSPACE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    RecArgs a{};
    a.P = preact; a.params = params; a.state = state; a.cu = cu_seqlens;
    a.rows = static_cast<int>(rows); a.T = T; a.d = static_cast<int>(d_h);
    a.H = H; a.gH = gH; a.g_last = g_last; a.gP = gP; a.g_state = g_state;
    a.part = static_cast<float *>(workspace);
    if (rows > 0) {
        const dim3 grid(static_cast<unsigned>((d_h + SEQ_THREADS - 1) / SEQ_THREADS), static_cast<unsigned>(rows < 65535 ? rows : 65535));
        if (dtype == NRNN_BF16) k_backward<__nv_bfloat16><<<grid, SEQ_THREADS, 0, s>>>(a);
        else k_backward<float><<<grid, SEQ_THREADS, 0, s>>>(a);
    }
    const int m = static_cast<int>(3 * d_h);
    k_join<<<(m + 127) / 128, 128, 0, s>>>(a.part, a.rows, m, gparams);
    return cudaGetLastError() == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

int nrnn_linear_recurrence_step(const void *preact, int dtype, const float *params, int64_t slots,
                                int64_t d_h, const float *state, void *h, float *state_out,
                                void *stream) {
    const int st = check(preact, dtype, params, slots, 1, d_h, nullptr, 0);
    if (st != NRNN_OK) return st;
    const int64_t es = dtype == NRNN_BF16 ? 2 : 4, n = slots * d_h;
    if (n == 0) return NRNN_OK;
    if (h == nullptr || state_out == nullptr || !aligned16(h) || !aligned16(state_out) || !aligned16(state) ||
        overlap(preact, 3 * n * es, h, n * es) || overlap(preact, 3 * n * es, state_out, 4 * n) ||
        overlap(h, n * es, state_out, 4 * n) || overlap(h, n * es, state, 4 * n) ||
        (state != state_out && overlap(state, 4 * n, state_out, 4 * n)))
        return NRNN_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t blocks = (n + 255) / 256;
    if (blocks > INT32_MAX) return NRNN_ERR_UNSUPPORTED;
    if (dtype == NRNN_BF16)
        k_step<<<static_cast<unsigned>(blocks), 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(preact), params, state, n,
                                                             static_cast<int>(d_h), static_cast<__nv_bfloat16 *>(h), state_out);
    else
        k_step<<<static_cast<unsigned>(blocks), 256, 0, s>>>(static_cast<const float *>(preact), params, state, n,
                                                             static_cast<int>(d_h), static_cast<float *>(h), state_out);
    return cudaGetLastError() == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

}  // extern "C"
