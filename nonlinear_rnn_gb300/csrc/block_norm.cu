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
//   gw_pre = sum gu x^,  gscale = w_post s,  gw_post = scale s,  s = sum t silu(gate) h^
//
// scale and w_post only ever act as their product, so the kernels hold that.
//
// (h silu(gate) is formed before the division by h's norm: preactivations and states
// whose product passes fp32's largest value, of about 1e19 each, overflow where the
// order above would not.)
//
// Neither direction has a product to speak of: both are bound by HBM, 5 row
// passes forward (x, h, gate in; x', u out) and 8 backward (x', h, gate, gx',
// gu in; gx, gh, ggate out).  A row is read once and stays in registers; the
// statistics are recomputed in the backward from the row it reads anyway
// instead of being stored.  All arithmetic and all sums are fp32.
//
// Measured: forward of 262144 x 1024 bf16 415 us (6.5 TB/s, 0.97 of a plain copy),
// backward of 65536 x 1024 bf16 188 us (5.7 TB/s), of 32768 x 256 fp32 55 us with
// the join (4.9 TB/s), of 65537 x 515 bf16 without a gate 161 us (2.5 TB/s: 66 pieces
// on 96 threads, and the rows' ends).
#include "../../include/nrnn.h"
#include "nrnn_device.cuh"
#include "nrnn_internal.h"
#include "rows.cuh"

namespace nrnn {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int MAX_D = 8192;   // a row in the registers of one CTA

// sigmoid of both lanes
__device__ __forceinline__ float2 sigmoid2(float2 v) {
    const float2 t = mul2(v, make_float2(-LOG2E, -LOG2E));
    const float2 d = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), make_float2(1.f, 1.f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }


struct NormArgs {
    const void *x, *h, *gate;            // x: x' in the backward
    const float *w_post, *scale, *w_pre; // null: ones
    const void *g_x, *g_u;               // backward: null = zeros
    void *out_x, *out_u;                 // forward: x', u
    void *gx, *gh, *g_gate;
    float *part;                         // backward: [CTAs][2][d] sums s and gw_pre
    int64_t rows;
    int d;
    float eps;
    int team_shift;                      // rows of up to a warp: log2 of the threads a row
    bool norm_u;                         // u is wanted (forward), w_pre's branch exists (backward)
};

// How a row lies in registers, for both directions.  TPR threads (a team) hold a
// row, as PIECES pieces of 16 bytes a thread, TPR pieces apart.  A team takes
// every teams-th row; the number of teams is a multiple of 8, so all rows of a
// team begin at the same place within a 16-byte piece even where d is odd: piece 0
// holds that many columns of the row before (`shift`), and the row's two end pieces
// are masked, and written by elements.  So a thread's columns are the same in
// all its rows, and the sums of the weights' gradients stay in its registers.
// EDGE: d is not a multiple of VEC, so a row has ends.  VEC = 1 (a piece is two
// elements): tensors that do not share an alignment.  (Odd rows read by elements
// took 446 us for the backward of 65537 x 515 bf16.)  The arithmetic is on pairs:
// one issue slot for two fp32 operations, since with bf16 storage the issue rate
// is nearer than the memory's.
template <typename T, int VEC_, int PIECES_, bool EDGE_> struct Layout {
    using Type = T;
    static constexpr int VEC = VEC_, PIECES = PIECES_;
    static constexpr bool EDGE = EDGE_;
    static constexpr int N = VEC * PIECES, PAIRS = N / 2;   // columns of a thread
};

// bytes < 16: the rest is zeros
__device__ __forceinline__ void copy_async_16(void *dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes)
                 : "memory");
}

template <typename L> struct Row {
    using T = typename L::Type;
    using P = Pack<T, L::VEC>;
    int c0[L::PIECES];   // first column of each piece (negative in a shifted row's first)
    bool whole[L::PIECES];
    uint32_t mask[L::EDGE ? L::PIECES * 4 : 1];   // bits of the pieces' words inside the row
    int d;
    int64_t total;       // elements of the array

    __device__ __forceinline__ Row(int t, int tpr, int d_, int shift, int64_t rows) : d(d_), total(rows * d_) {
#pragma unroll
        for (int i = 0; i < L::PIECES; ++i) {
            c0[i] = (t + i * tpr) * L::VEC - shift;
            whole[i] = L::EDGE ? c0[i] >= 0 && c0[i] + L::VEC <= d : c0[i] < d;
            if (L::EDGE) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    constexpr int PER = 4 / sizeof(T);
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < PER; ++e) {
                        const int c = c0[i] + w * PER + e;
                        if (c >= 0 && c < d) m |= PER == 1 ? 0xffffffffu : 0xffffu << (16 * e);
                    }
                    mask[(i * 4 + w) % (L::EDGE ? L::PIECES * 4 : 1)] = m;
                }
            }
        }
    }
    // starts the copy of this thread's pieces to shared memory, THREADS pieces apart
    template <int THREADS>
    __device__ __forceinline__ void fetch(const void *base, int64_t at, P *to) const {
        const T *p = static_cast<const T *>(base) + at;
#pragma unroll
        for (int i = 0; i < L::PIECES; ++i) {
            P *dst = to + i * THREADS;
            if (c0[i] >= d) continue;
            if (L::EDGE) {
                // an end piece is copied whole too, but for what lies past the array
                const int64_t left = (total - at - c0[i]) * static_cast<int64_t>(sizeof(T));
                copy_async_16(dst, p + c0[i], left < 16 ? static_cast<int>(left) : 16);
            } else if (sizeof(P) == 16) {
                copy_async_16(dst, p + c0[i], 16);
            } else {
                *dst = *reinterpret_cast<const P *>(p + c0[i]);
            }
        }
    }
    __device__ __forceinline__ void store(void *base, int64_t at, const float2 (&f)[L::PAIRS]) const {
        T *p = static_cast<T *>(base) + at;
#pragma unroll
        for (int i = 0; i < L::PIECES; ++i) {
            P o;
            narrow(f, i, o);
            if (whole[i]) {
                *reinterpret_cast<P *>(p + c0[i]) = o;
            } else if (L::EDGE) {   // by words, and the one that holds the row's end by elements
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    constexpr int PER = 4 / sizeof(T);
                    const uint32_t m = mask[(i * 4 + w) % (L::EDGE ? L::PIECES * 4 : 1)];
                    T *to = p + c0[i] + w * PER;
                    if (m == 0xffffffffu) *reinterpret_cast<uint32_t *>(to) = reinterpret_cast<const uint32_t *>(&o)[w];
                    else if (PER == 2 && m == 0xffffu) to[0] = o.v[(w * PER) % L::VEC];
                    else if (PER == 2 && m == 0xffff0000u) to[1] = o.v[(w * PER + 1) % L::VEC];
                }
            }
        }
    }
    // the pieces as fp32, zeros outside the row
    template <int THREADS>
    __device__ __forceinline__ void widen(const P *from, float2 (&f)[L::PAIRS]) const {
#pragma unroll
        for (int i = 0; i < L::PIECES; ++i) {
            P v{};
            if (L::EDGE || whole[i]) v = from[i * THREADS];
            if (L::EDGE) {   // not the neighbouring rows' columns
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    reinterpret_cast<uint32_t *>(&v)[w % (sizeof(P) / 4 > 0 ? sizeof(P) / 4 : 1)] &=
                        mask[(i * 4 + w) % (L::EDGE ? L::PIECES * 4 : 1)];
            }
            if constexpr (sizeof(T) == 2 && L::VEC > 1) {
#pragma unroll
                for (int e = 0; e < L::VEC / 2; ++e) {   // a bf16 is the upper half of its fp32
                    const uint32_t w = reinterpret_cast<const uint32_t *>(&v)[e];
                    f[i * (L::VEC / 2) + e] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
                }
            } else {
#pragma unroll
                for (int e = 0; e < L::VEC; ++e) {
                    const int j = i * L::VEC + e;
                    (j % 2 == 0 ? f[j / 2].x : f[j / 2].y) = to_f32(v.v[e]);
                }
            }
        }
    }
    static __device__ __forceinline__ void narrow(const float2 (&f)[L::PAIRS], int i, P &o) {
        if constexpr (sizeof(T) == 2 && L::VEC > 1) {
#pragma unroll
            for (int e = 0; e < L::VEC / 2; ++e) {
                const float2 v = f[i * (L::VEC / 2) + e];
                reinterpret_cast<__nv_bfloat162 *>(&o)[e] = __floats2bfloat162_rn(v.x, v.y);
            }
        } else {
#pragma unroll
            for (int e = 0; e < L::VEC; ++e) {
                const int j = i * L::VEC + e;
                o.v[e] = from_f32<T>(j % 2 == 0 ? f[j / 2].x : f[j / 2].y);
            }
        }
    }
    // zero outside the row
    __device__ __forceinline__ float column(const float *a, const float *b, int j) const {
        const int c = c0[j / L::VEC] + j % L::VEC;
        if (c < 0 || c >= d) return 0.f;
        return (a == nullptr ? 1.f : __ldg(a + c)) * (b == nullptr ? 1.f : __ldg(b + c));
    }
};

// TPR = 32: up to a warp a row (a power of two, 1 << shift) and several rows a CTA;
// else up to TPR threads, a CTA
template <int TPR> struct Teams {
    static constexpr int THREADS = TPR <= 32 ? 128 : TPR;
    int t, tpr, in_cta, per_cta, team, teams;
    __device__ __forceinline__ Teams(int shift) {
        tpr = TPR <= 32 ? 1 << shift : blockDim.x;
        per_cta = TPR <= 32 ? THREADS >> shift : 1;
        in_cta = TPR <= 32 ? threadIdx.x >> shift : 0;
        t = TPR <= 32 ? threadIdx.x & (tpr - 1) : threadIdx.x;
        team = blockIdx.x * per_cta + in_cta;
        teams = gridDim.x * per_cta;
    }
};

// This thread's columns of scale w_post and of w_pre (null: ones; zeros outside the
// row) wait in shared memory, in an order that only this thread reads: in
// registers they would cost what keeps the next row's loads in flight.
template <typename L, int THREADS> struct Weights {
    float4 *mine;
    static constexpr int QUADS = L::N / 4;
    static constexpr size_t BYTES = sizeof(float) * 2 * L::N * THREADS;

    __device__ __forceinline__ Weights(float4 *smem, const Row<L> &r, const NormArgs &a)
        : mine(smem + threadIdx.x) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int q = 0; q < QUADS; ++q) {
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f[e] = w == 0 ? r.column(a.w_post, a.scale, 4 * q + e) : r.column(a.w_pre, nullptr, 4 * q + e);
                mine[(w * QUADS + q) * THREADS] = make_float4(f[0], f[1], f[2], f[3]);
            }
    }
    // volatile: not to be kept in registers across the loop after all
    __device__ __forceinline__ void load(int w, float2 (&f)[L::PAIRS]) const {
#pragma unroll
        for (int q = 0; q < QUADS; ++q)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(f[2 * q].x), "=f"(f[2 * q].y), "=f"(f[2 * q + 1].x), "=f"(f[2 * q + 1].y)
                         : "r"(smem_u32(mine + (w * QUADS + q) * THREADS)));
    }
};
enum { W_OUT = 0, W_PRE = 1 };

// Rows on their way: each thread copies its own pieces to its own places in shared
// memory (cp.async) and reads them back itself, so the next row's loads are in
// flight over this row's sums without registers or barriers.  (Loads to registers
// a row ahead were waited for at once: 327 us for the backward of 65536 x 1024
// bf16, and 237 us without looking ahead.)
template <typename L, int THREADS, int TENSORS, int DEPTH> struct Stage {
    using P = typename Row<L>::P;
    P *mine;
    static constexpr size_t BYTES = sizeof(P) * L::PIECES * TENSORS * DEPTH * THREADS;
    __device__ __forceinline__ explicit Stage(void *smem) : mine(static_cast<P *>(smem) + threadIdx.x) {}
    __device__ __forceinline__ P *at(int turn, int tensor) const {
        return mine + (turn * TENSORS + tensor) * (L::PIECES * THREADS);
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait_row() {   // the oldest row has arrived
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    }
};
// rows in flight: wide rows leave room for one
constexpr int depth_for(int tpr) { return tpr > 512 ? 1 : 2; }
template <typename L, int TPR, int TENSORS> constexpr size_t smem_for() {
    return Weights<L, Teams<TPR>::THREADS>::BYTES + Stage<L, Teams<TPR>::THREADS, TENSORS, depth_for(TPR)>::BYTES;
}

// N sums over a team.  A team of more than a warp is a CTA: buf is [N][32], and
// the caller alternates between two of them, so one barrier a call is enough.
template <int TPR, int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float *buf, int tpr) {
    if (TPR <= 32) {
        for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(FULL_MASK, v[i], o);
        return;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(FULL_MASK, v[i], o);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i * 32 + (threadIdx.x >> 5)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.f;
        if (TPR <= 128) {
#pragma unroll
            for (int w = 0; w < 4; ++w) s += w < warps ? buf[i * 32 + w] : 0.f;
        } else {
            for (int w = 0; w < warps; ++w) s += buf[i * 32 + w];
        }
        v[i] = s;
    }
}

// resident threads an SM that the kernels' registers and shared memory leave room for
constexpr int FWD_THREADS_PER_SM = 640;
// backward: by a thread's columns; fp32 rows (vec = 4) stage twice the bytes
constexpr int bwd_threads_per_sm(int vec, int columns) {
    return columns > 8 ? 384 : vec == 8 ? 640 : 512;
}
constexpr int resident(int threads, int per_sm) { return per_sm / threads > 0 ? per_sm / threads : 1; }

// ------------------------------------------------------------------- forward
template <typename L, int TPR>
__global__ void __launch_bounds__(Teams<TPR>::THREADS, resident(Teams<TPR>::THREADS, FWD_THREADS_PER_SM))
    k_norm_forward(const NormArgs a) {
    extern __shared__ float4 norm_smem[];
    __shared__ float red[2][2 * 32];
    wait_for_prerequisites();
    const Teams<TPR> g(a.team_shift);
    const Row<L> r(g.t, g.tpr, a.d, static_cast<int>(static_cast<int64_t>(g.team) * a.d % L::VEC), a.rows);
    const float inv_d = 1.f / a.d;
    const Weights<L, Teams<TPR>::THREADS> weights(norm_smem, r, a);
    constexpr int THREADS = Teams<TPR>::THREADS, DEPTH = depth_for(TPR);
    const Stage<L, THREADS, 3, DEPTH> stage(reinterpret_cast<unsigned char *>(norm_smem) +
                                            Weights<L, THREADS>::BYTES);
    auto fetch_row = [&](int64_t row, int turn) {
        if (row < a.rows) {
            const int64_t at = row * a.d;
            r.template fetch<THREADS>(a.x, at, stage.at(turn, 0));
            if (a.h != nullptr) r.template fetch<THREADS>(a.h, at, stage.at(turn, 1));
            if (a.gate != nullptr) r.template fetch<THREADS>(a.gate, at, stage.at(turn, 2));
        }
        stage.commit();
    };
    // teams that share a warp run the same number of rounds
    const int64_t rounds = (a.rows + g.teams - 1) / g.teams;
    int64_t row = g.team;
    if (DEPTH > 1) fetch_row(row, 0);
    for (int64_t i = 0; i < rounds; ++i, row += g.teams) {
        const int turn = DEPTH > 1 ? i & 1 : 0;
        fetch_row(DEPTH > 1 ? row + g.teams : row, DEPTH > 1 ? turn ^ 1 : 0);
        stage.wait_row();
        float2 x[L::PAIRS], w[L::PAIRS];
        r.template widen<THREADS>(stage.at(turn, 0), x);
        const int64_t at = row * a.d;
        if (a.h != nullptr) {
            float2 v[L::PAIRS], ss = both(0.f);
            r.template widen<THREADS>(stage.at(turn, 1), v);
#pragma unroll
            for (int e = 0; e < L::PAIRS; ++e) ss = fma2(v[e], v[e], ss);
            if (a.gate != nullptr) {
                float2 gate[L::PAIRS];
                r.template widen<THREADS>(stage.at(turn, 2), gate);
#pragma unroll
                for (int e = 0; e < L::PAIRS; ++e)
                    v[e] = mul2(v[e], mul2(gate[e], sigmoid2(gate[e])));
            }
            float sum[1] = {ss.x + ss.y};
            team_sums<TPR, 1>(sum, red[i & 1], g.tpr);
            const float2 q = both(rsqrtf(sum[0] * inv_d + a.eps));
            weights.load(W_OUT, w);
#pragma unroll
            for (int e = 0; e < L::PAIRS; ++e) x[e] = fma2(mul2(v[e], q), w[e], x[e]);
            if (row < a.rows) r.store(a.out_x, at, x);
        }
        if (!a.norm_u) continue;
        float2 ss = both(0.f);
#pragma unroll
        for (int e = 0; e < L::PAIRS; ++e) ss = fma2(x[e], x[e], ss);
        float sum[1] = {ss.x + ss.y};
        team_sums<TPR, 1>(sum, red[i & 1] + 32, g.tpr);
        const float2 s = both(rsqrtf(sum[0] * inv_d + a.eps));
        weights.load(W_PRE, w);
#pragma unroll
        for (int e = 0; e < L::PAIRS; ++e) x[e] = mul2(mul2(x[e], s), w[e]);
        if (row < a.rows) r.store(a.out_u, at, x);
    }
}

// ------------------------------------------------------------------ backward
template <typename L, int TPR>
__global__ void __launch_bounds__(Teams<TPR>::THREADS, resident(Teams<TPR>::THREADS, bwd_threads_per_sm(L::VEC, L::N)))
    k_norm_backward(const NormArgs a) {
    __shared__ float red[2][4 * 32];   // three sums, then one; two rows in turn
    extern __shared__ float4 norm_smem[];
    const Teams<TPR> g(a.team_shift);
    dependents_may_launch();
    wait_for_prerequisites();
    const Row<L> r(g.t, g.tpr, a.d, static_cast<int>(static_cast<int64_t>(g.team) * a.d % L::VEC), a.rows);
    const float inv_d = 1.f / a.d;
    const Weights<L, Teams<TPR>::THREADS> weights(norm_smem, r, a);
    float2 s_out[L::PAIRS] = {}, s_pre[L::PAIRS] = {};
    constexpr int THREADS = Teams<TPR>::THREADS, DEPTH = depth_for(TPR);
    const Stage<L, THREADS, 5, DEPTH> stage(reinterpret_cast<unsigned char *>(norm_smem) +
                                            Weights<L, THREADS>::BYTES);
    auto fetch_row = [&](int64_t row, int turn) {
        if (row < a.rows) {
            const int64_t at = row * a.d;
            if (a.norm_u) {
                r.template fetch<THREADS>(a.x, at, stage.at(turn, 0));
                r.template fetch<THREADS>(a.g_u, at, stage.at(turn, 1));
            }
            if (a.g_x != nullptr) r.template fetch<THREADS>(a.g_x, at, stage.at(turn, 2));
            if (a.h != nullptr) r.template fetch<THREADS>(a.h, at, stage.at(turn, 3));
            if (a.gate != nullptr) r.template fetch<THREADS>(a.gate, at, stage.at(turn, 4));
        }
        stage.commit();
    };
    const int64_t rounds = (a.rows + g.teams - 1) / g.teams;
    int64_t row = g.team;
    if (DEPTH > 1) fetch_row(row, 0);
    for (int64_t i = 0; i < rounds; ++i, row += g.teams) {
        const int turn = DEPTH > 1 ? i & 1 : 0;
        fetch_row(DEPTH > 1 ? row + g.teams : row, DEPTH > 1 ? turn ^ 1 : 0);
        stage.wait_row();
        const bool live = row < a.rows;   // a team past the end adds nothing
        float2 x[L::PAIRS] = {}, h[L::PAIRS] = {}, gx[L::PAIRS] = {}, gu[L::PAIRS] = {};
        if (live) {
            if (a.norm_u) {
                r.template widen<THREADS>(stage.at(turn, 0), x);
                r.template widen<THREADS>(stage.at(turn, 1), gu);
            }
            if (a.g_x != nullptr) r.template widen<THREADS>(stage.at(turn, 2), gx);
            if (a.h != nullptr) r.template widen<THREADS>(stage.at(turn, 3), h);
        }
        const int64_t at = row * a.d;
        float2 m0 = both(0.f), m1 = m0, m2 = m0, w[L::PAIRS];
        weights.load(W_PRE, w);
#pragma unroll
        for (int e = 0; e < L::PAIRS; ++e) {
            m0 = fma2(x[e], x[e], m0);
            w[e] = mul2(gu[e], w[e]);   // a
            m1 = fma2(w[e], x[e], m1);
            m2 = fma2(h[e], h[e], m2);
        }
        float m[3] = {m0.x + m0.y, m1.x + m1.y, m2.x + m2.y};
        team_sums<TPR, 3>(m, red[i & 1], g.tpr);
        if (a.norm_u && live) {
            const float s = rsqrtf(m[0] * inv_d + a.eps);
            const float2 s2 = both(s), mean_ax = both(-m[1] * inv_d * s);   // -<a x^>
#pragma unroll
            for (int e = 0; e < L::PAIRS; ++e) {
                const float2 xn = mul2(x[e], s2);
                s_pre[e] = fma2(gu[e], xn, s_pre[e]);
                gx[e] = fma2(s2, fma2(xn, mean_ax, w[e]), gx[e]);   // t
            }
        }
        if (live) r.store(a.gx, at, gx);
        if (a.h == nullptr) continue;
        const float q = rsqrtf(m[2] * inv_d + a.eps);
        float2 k2 = both(0.f);
        if (live) {
            weights.load(W_OUT, w);
            float2 gate[L::PAIRS] = {};
            if (a.gate != nullptr) r.template widen<THREADS>(stage.at(turn, 4), gate);
#pragma unroll
            for (int e = 0; e < L::PAIRS; ++e) {
                h[e] = mul2(h[e], both(q));                     // h^
                const float2 c = mul2(gx[e], w[e]);             // t scale w_post
                if (a.gate != nullptr) {
                    const float2 sg = sigmoid2(gate[e]);
                    const float2 of = mul2(gate[e], sg);        // silu
                    // silu' = sg (1 + gate (1 - sg)) = sg + of - of sg
                    const float2 slope = fma2(of, make_float2(-sg.x, -sg.y), add2(sg, of));
                    gate[e] = mul2(mul2(c, h[e]), slope);
                    s_out[e] = fma2(mul2(gx[e], of), h[e], s_out[e]);
                    gx[e] = mul2(c, of);                        // b
                } else {
                    s_out[e] = fma2(gx[e], h[e], s_out[e]);
                    gx[e] = c;
                }
                k2 = fma2(gx[e], h[e], k2);
            }
            if (a.gate != nullptr) r.store(a.g_gate, at, gate);
        }
        float k[1] = {k2.x + k2.y};
        team_sums<TPR, 1>(k, red[i & 1] + 3 * 32, g.tpr);
        const float2 mean_bh = both(-k[0] * inv_d), q2 = both(q);
#pragma unroll
        for (int e = 0; e < L::PAIRS; ++e) gx[e] = mul2(q2, fma2(h[e], mean_bh, gx[e]));
        if (live) r.store(a.gh, at, gx);
    }
    // this CTA's sums: its teams in order, then to the workspace
    float *part = a.part + blockIdx.x * static_cast<int64_t>(2) * a.d;
    float *join = reinterpret_cast<float *>(norm_smem);   // [2][d], where the weights were
    for (int o = 0; o < g.per_cta; ++o) {
        if (TPR <= 32) __syncthreads();
        if (g.in_cta != o) continue;
        float *to = o < g.per_cta - 1 ? join : part;
#pragma unroll
        for (int j = 0; j < L::N; ++j) {
            const int c = r.c0[j / L::VEC] + j % L::VEC;
            if (c < 0 || c >= a.d) continue;
            float v[2] = {j % 2 == 0 ? s_out[j / 2].x : s_out[j / 2].y,
                          j % 2 == 0 ? s_pre[j / 2].x : s_pre[j / 2].y};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (TPR <= 32 && o > 0) v[q] += join[q * a.d + c];
                to[q * a.d + c] = v[q];
            }
        }
    }
}

// sums of the CTAs' partial sums, in order: a warp's lanes take 32 columns, the
// warps of the CTA every JOIN_WARPS-th partial
constexpr int JOIN_WARPS = 16;

__global__ void __launch_bounds__(JOIN_WARPS * 32)
    k_norm_join(const float *__restrict__ part, int n_part, int d, const float *w_post,
                const float *scale, float *gw_post, float *g_scale, float *gw_pre) {
    __shared__ float sum[JOIN_WARPS][32];
    wait_for_prerequisites();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;   // column of [2][d]
    float s = 0.f;
    if (c < 2 * d) {
#pragma unroll 8
        for (int p = w; p < n_part; p += JOIN_WARPS) s += part[static_cast<int64_t>(p) * 2 * d + c];
    }
    sum[w][lane] = s;
    __syncthreads();
    if (w > 0 || c >= 2 * d) return;
#pragma unroll
    for (int q = 1; q < JOIN_WARPS; ++q) s += sum[q][lane];
    if (c < d) {
        if (gw_post != nullptr) gw_post[c] = scale == nullptr ? s : s * scale[c];
        if (g_scale != nullptr) g_scale[c] = w_post == nullptr ? s : s * w_post[c];
    } else if (gw_pre != nullptr) {
        gw_pre[c - d] = s;
    }
}

// ---------------------------------------------------------------- host side
bool aligned_to(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool all_aligned_to(size_t a, std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (!aligned_to(p, a)) return false;
    return true;
}

// Threads a row: the fewest that hold it in `pieces` each, a power of two up to
// a warp, whole warps beyond.
int team_size(int d, int vec, int pieces) {
    int common = vec;   // the largest power of two that divides both
    while (d % common != 0) common /= 2;
    const int have = (d + vec - common + vec - 1) / vec;   // pieces of the most shifted row
    const int need = (have + pieces - 1) / pieces;
    if (need > 32) return (need + 31) / 32 * 32;
    int t = 1;
    while (t < need) t *= 2;
    return t;
}
// CTAs: enough teams for every row once, at most the resident ones; a multiple of
// 8 teams
int cta_count(int64_t rows, int tpr, int threads_per_sm) {
    const int64_t per = tpr <= 32 ? 128 / tpr : 1;
    const int threads = tpr <= 32 ? 128 : tpr;
    int64_t most = 152 * resident(threads, threads_per_sm);
    const int64_t want = (rows + per - 1) / per;
    most = want < most ? want : most;
    return static_cast<int>(per >= 8 ? most : (most * per + 7) / 8 * 8 / per);
}

template <typename L, int TPR, int TENSORS, typename K>
cudaError_t launch_norm(K kernel, NormArgs a, int ctas, int tpr, cudaStream_t s) {
    constexpr size_t smem = smem_for<L, TPR, TENSORS>();
    if (smem > 40 * 1024) {   // 48 KB with the static part need no attribute
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    while (TPR <= 32 && (1 << a.team_shift) < tpr) ++a.team_shift;
    return launch_dependent(kernel, ctas, TPR <= 32 ? Teams<TPR>::THREADS : tpr, smem, s, a);
}

// Pieces a thread forward: two.  A bf16 row that two pieces a thread would leave half empty takes
// one forward (65537 x 515: 66 pieces in 3 warps instead of 128 in 2).
template <typename T, int VEC, bool EDGE, int PIECES>
cudaError_t forward_as(const NormArgs &a, cudaStream_t s) {
    using L = Layout<T, VEC, PIECES, EDGE>;
    const int tpr = team_size(a.d, VEC, PIECES), ctas = cta_count(a.rows, tpr, FWD_THREADS_PER_SM);
    if (tpr <= 32) return launch_norm<L, 32, 3>(k_norm_forward<L, 32>, a, ctas, tpr, s);
    if (tpr <= 128) return launch_norm<L, 128, 3>(k_norm_forward<L, 128>, a, ctas, tpr, s);
    if (tpr <= 512) return launch_norm<L, 512, 3>(k_norm_forward<L, 512>, a, ctas, tpr, s);
    return launch_norm<L, 1024, 3>(k_norm_forward<L, 1024>, a, ctas, tpr, s);
}

template <typename T, int VEC, bool EDGE> cudaError_t forward_for(const NormArgs &a, cudaStream_t s) {
    if constexpr (VEC == 1) return forward_as<T, 1, false, 8>(a, s);
    else if constexpr (VEC == 8) {
        if (team_size(a.d, VEC, 1) < 2 * team_size(a.d, VEC, 2)) return forward_as<T, VEC, EDGE, 1>(a, s);
    }
    if constexpr (VEC > 1) return forward_as<T, VEC, EDGE, 2>(a, s);
}

// Backward: 8 columns a thread; a bf16 row of 33 to 64 pieces takes a warp with two
// pieces a thread instead of two warps, without barriers and with the work that does
// not grow with the columns done once (65536 x 512 127 -> 104 us; with three pieces
// the registers leave too few warps: 65537 x 515 201 -> 232 us).
struct BwdShape { int pieces, tpr; };
BwdShape bwd_shape(int d, int vec) {
    if (vec == 8 && team_size(d, vec, 1) > 32 && team_size(d, vec, 2) <= 32) return {2, team_size(d, vec, 2)};
    return {8 / vec, team_size(d, vec, 8 / vec)};
}

template <typename T, int VEC, bool EDGE>
cudaError_t backward_for(const NormArgs &a, int ctas, cudaStream_t s) {
    const BwdShape shape = bwd_shape(a.d, VEC);
    const int tpr = shape.tpr;
    if constexpr (VEC == 8) {
        using L2 = Layout<T, VEC, 2, EDGE>;
        if (shape.pieces == 2) return launch_norm<L2, 32, 5>(k_norm_backward<L2, 32>, a, ctas, tpr, s);
    }
    using L = Layout<T, VEC, 8 / VEC, EDGE>;
    if (tpr <= 32) return launch_norm<L, 32, 5>(k_norm_backward<L, 32>, a, ctas, tpr, s);
    if (tpr <= 128) return launch_norm<L, 128, 5>(k_norm_backward<L, 128>, a, ctas, tpr, s);
    if (tpr <= 512) return launch_norm<L, 512, 5>(k_norm_backward<L, 512>, a, ctas, tpr, s);
    return launch_norm<L, 1024, 5>(k_norm_backward<L, 1024>, a, ctas, tpr, s);
}

// calls f<T, VEC, EDGE>(args...) for the storage type, the access width and d
#define NRNN_BY_ROW(dtype, vec, d, f, ...)                                            \
    ((dtype) == NRNN_BF16 ? ((vec) == 1          ? f<__nv_bfloat16, 1, false>(__VA_ARGS__) \
                             : (d) % (vec) == 0  ? f<__nv_bfloat16, 8, false>(__VA_ARGS__) \
                                                 : f<__nv_bfloat16, 8, true>(__VA_ARGS__)) \
                          : ((vec) == 1          ? f<float, 1, false>(__VA_ARGS__)         \
                             : (d) % (vec) == 0  ? f<float, 4, false>(__VA_ARGS__)         \
                                                 : f<float, 4, true>(__VA_ARGS__)))

// CTAs of a backward launch
int backward_ctas(int64_t rows, int d, int vec) {
    const BwdShape shape = bwd_shape(d, vec);
    return cta_count(rows, shape.tpr, bwd_threads_per_sm(vec, shape.pieces * vec));
}

int check_norm(int dtype, int64_t rows, int64_t d, float eps) {
    if (dtype != NRNN_F32 && dtype != NRNN_BF16) return NRNN_ERR_INVALID_ARG;
    if (rows < 0 || d <= 0 || !(eps >= 0.f)) return NRNN_ERR_INVALID_ARG;
    if (d > MAX_D) return NRNN_ERR_UNSUPPORTED;
    return NRNN_OK;
}

// 16-byte pieces where every tensor begins on a 16-byte boundary, else one element
// (a row of 8192 odd columns would take more than a CTA's threads with pieces)
int width_for(int elem, int64_t d, std::initializer_list<const void *> ptrs) {
    const int vec = 16 / elem;
    if (team_size(static_cast<int>(d), vec, 8 / vec) > 1024) return 1;
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
    if (!all_aligned_to(elem, {x, h, gate, x_out, u}) ||
        !all_aligned_to(sizeof(float), {w_post, scale, w_pre}))
        return NRNN_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = x; a.h = h; a.gate = gate;
    a.w_post = w_post; a.scale = scale; a.w_pre = w_pre;
    a.out_x = x_out; a.out_u = u;
    a.rows = rows; a.d = static_cast<int>(d); a.eps = eps;
    a.norm_u = u != nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int vec = width_for(elem, d, {x, h, gate, x_out, u});
    const cudaError_t e = NRNN_BY_ROW(dtype, vec, d, forward_for, a, s);
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

size_t nrnn_block_norm_backward_workspace_bytes(int64_t rows, int64_t d) {
    if (rows < 0 || d <= 0 || d > MAX_D) return 0;
    int ctas = 1;
    if (rows > 0)
        for (int vec : {1, 4, 8}) {
            const int n = backward_ctas(rows, static_cast<int>(d), vec);
            ctas = n > ctas ? n : ctas;
        }
    const size_t bytes = sizeof(float) * 2 * d * ctas;
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
    if (!all_aligned_to(elem, {x_out, h, gate, g_x, g_u, gx, gh, g_gate}) ||
        !all_aligned_to(sizeof(float), {w_post, scale, w_pre, gw_post, g_scale, gw_pre}))
        return NRNN_ERR_INVALID_ARG;
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
    int ctas = 0;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        const int vec = width_for(elem, d, {x_out, h, gate, g_x, g_u, gx, gh, g_gate});
        ctas = backward_ctas(rows, a.d, vec);
        e = NRNN_BY_ROW(dtype, vec, d, backward_for, a, ctas, s);
    }
    if (e == cudaSuccess) {
        e = launch_dependent(k_norm_join, (2 * a.d + 31) / 32, JOIN_WARPS * 32, 0, s, a.part, ctas, a.d,
                             w_post, scale, gw_post, g_scale, gw_pre);
    }
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

}  // extern "C"
