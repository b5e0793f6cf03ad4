// Softmax cross entropy over a vocabulary, in pieces of the vocabulary, without
// keeping the logits, and its gradient.
//
//   z_iv = c <x_i, W_v>,  lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_i,t(i)
//   G_iv = gl_i c (exp(z_iv - lse_i) - [v = t(i)]),  gx = G W,  gW = G^T x
//
// 2 N V d operations forward, 6 N V d backward (the logits are computed again):
// bound by the tensor cores, except for few rows, where reading W bounds it.
//
// All three products run on one persistent tcgen05 kernel (k_vocab_gemm): one
// CTA per SM, 128 x (up to 256) tiles, TMA into a ring of 128-byte-swizzled
// stages, one thread issuing tcgen05.mma into one of two TMEM accumulators
// while the epilogue warps drain the other.  Its forms differ in the operands'
// orientation (the transposed ones are read MN-major from where they lie: no
// transposed copy is made) and in the epilogue:
//   LSE  x W^T   running maximum and sum of each row over the unit's vocabulary
//   DL   x W^T   G of one piece of the vocabulary, to the workspace
//   GX   G W     gx, or its share of this piece / this split of the piece
//   GW   G^T x   rows of gW of this piece
// The piece of G is all that is ever kept of the N x V matrix.
//
// Rows whose target is ignored take no part: the kept rows are numbered on the
// device and gathered (k_kept_rows, k_gather_rows), and the kernel reads their
// number there, so ignored rows cost nothing and whatever they hold (infinities,
// NaN) reaches no output.
//
// fp32 inputs are written as three bf16 planes, v = hi + mid + lo exactly up to
// 2^-24, and a product is the six plane products down to 2^-16 relative:
// (lo,hi) (mid,mid) (hi,lo) (mid,hi) (hi,mid) (hi,hi).  The tensor cores'
// accumulation rounds coarser than fp32 addition does, so an accumulator takes
// at most 512 elements of the inner dimension before the epilogue adds it to
// fp32 registers.
//
// Every wait is bounded.  One that gives up sets g_vocab_error and the CTA's
// abort flag, which ends the other roles' waits too: the producer and the issuer
// stop (and see their copies and products in flight through), and the epilogue
// writes NaN from there on.
#include "../../include/nrnn.h"
#include "nrnn_device.cuh"
#include "nrnn_internal.h"
#include "rows.cuh"
#include "tcgen05.cuh"

namespace nrnn {
namespace {

constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int SMS = 152;   // work is divided for this many persistent CTAs

__device__ uint32_t g_vocab_error;

enum Form { LSE, DL, GX, GW };

constexpr int BM = 128, BN = 256, BK = 64, STAGES = 4;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 4;
constexpr int GEMM_THREADS = 128 + EPI_WARPS * 32;
constexpr int BOX = 32;                                   // rows and columns of a stored block of G
constexpr int BOX_BYTES = BOX * BOX * 2;
constexpr size_t GEMM_SMEM = STAGES * STAGE_BYTES + EPI_WARPS * 2 * BOX_BYTES + 1024;
constexpr int SPLIT_BN = 128;      // fp32: columns of a tile (its sums are held in registers)
constexpr int SPLIT_CHUNK = 8;     // fp32: 64-wide slices per accumulator
constexpr int SEGMENTS = 6;        // fp32: plane products, smallest first
__device__ constexpr int PLANE_A[SEGMENTS] = {2, 1, 0, 1, 0, 0};
__device__ constexpr int PLANE_B[SEGMENTS] = {0, 1, 2, 0, 1, 0};

struct GemmArgs {
    const int *kept;          // device: number of kept rows
    int M;                    // rows of the product on the host's side: -1 = kept
    int K;                    // inner size: -1 = kept
    int bn;                   // columns of a tile: a multiple of 16, at most BN
    int n_cols;               // columns of the product (LSE, DL: of this piece)
    int col0;                 // LSE, DL: first vocabulary row; GX: B's first inner row;
                              // GW: first row of gW
    int group;                // LSE: column tiles a unit takes one after another
    int splits;               // GX: splits of the inner dimension
    float scale;              // logit scale c
    const int2 *row;          // per kept row {its row in x, its target}
    const float2 *grad;       // DL: per kept row {lse log2(e), gl c}
    float2 *part;             // LSE: [rows][groups] {maximum, sum} in base 2
    float *z_target;          // LSE: base-2 logit of the target
    void *out;                // GX, GW: the gradient in the storage type
    float *acc;               // GX: [splits][rows][acc_pitch] sums over pieces (null: store out)
    int64_t acc_plane;
    int acc_pitch;
    bool acc_add;             // GX: add to acc
    int d;                    // width of gx and gW rows
};

// mbar_wait_bounded that also ends when another role of the CTA gave up
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile uint32_t *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (*abort != 0) return false;
        if (mbar_try_wait_hint(bar, parity, 1000000u)) return true;
        if (globaltimer_ns() - t0 > WAIT_NS) {
            *abort = 1;
            atomicOr(&g_vocab_error, 2u);
            return false;
        }
    }
    return true;
}

template <typename T> __device__ __forceinline__ void store_cols(T *p, const float (&v)[32], int n, bool wide) {
    constexpr int VEC = 16 / sizeof(T);
    if (wide) {
#pragma unroll
        for (int c = 0; c < 32; c += VEC) {
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = v[c + e];
            if (c < n) store_f32<T, VEC>(p + c, o);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (c < n) p[c] = from_f32<T>(v[c]);
    }
}

// A unit is what a CTA takes at a time: a tile, or (LSE) `group` tiles beside
// one another.  Every role walks the same sequence of tiles and chunks.
template <int FORM> struct Walk {
    int tiles_m, tiles_n, n_units, kb;   // kb: 64-wide slices of the inner dimension
    __device__ Walk(const GemmArgs &a) {
        const int kept = *a.kept;
        const int M = a.M < 0 ? kept : a.M, K = a.K < 0 ? kept : a.K;
        tiles_m = (M + BM - 1) / BM;
        tiles_n = (a.n_cols + a.bn - 1) / a.bn;
        kb = (K + BK - 1) / BK;
        n_units = FORM == LSE  ? tiles_m * ((tiles_n + a.group - 1) / a.group)
                  : FORM == GX ? tiles_m * tiles_n * a.splits
                               : tiles_m * tiles_n;
    }
};
struct Unit { int m0, n0, tiles, k0, k1, split; };

template <int FORM>
__device__ __forceinline__ Unit unit_at(const Walk<FORM> &w, const GemmArgs &a, int u) {
    Unit t;
    t.k0 = 0; t.k1 = w.kb; t.tiles = 1; t.split = 0;
    if (FORM == LSE || FORM == DL) {
        // rows fastest: the CTAs working at one time share a tile of W
        t.m0 = u % w.tiles_m * BM;
        const int g = u / w.tiles_m;
        if (FORM == LSE) {
            t.n0 = g * a.group;
            t.tiles = w.tiles_n - t.n0 < a.group ? w.tiles_n - t.n0 : a.group;
            t.n0 *= a.bn;
        } else {
            t.n0 = g * a.bn;
        }
    } else {
        // columns fastest: they share G's tile
        t.n0 = u % w.tiles_n * a.bn;
        u /= w.tiles_n;
        t.m0 = u % w.tiles_m * BM;
        if (FORM == GX) {
            t.split = u / w.tiles_m;
            t.k0 = static_cast<int>(static_cast<int64_t>(w.kb) * t.split / a.splits);
            t.k1 = static_cast<int>(static_cast<int64_t>(w.kb) * (t.split + 1) / a.splits);
        }
    }
    return t;
}

// T: storage type of the inputs (float: split products)
template <int FORM, typename T>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    k_vocab_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmOut, const GemmArgs a) {
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr bool MN_A = FORM == GW, MN_B = FORM == GX || FORM == GW;
    constexpr uint32_t TMEM_COLS = 512;   // two accumulators
    extern __shared__ unsigned char dsmem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES], accf_bar[2], acce_bar[2],
        drain_bar;
    __shared__ uint32_t s_tmem;
    __shared__ volatile uint32_t s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 1);
            mbar_init(&acce_bar[b], EPI_WARPS * 32);
        }
        mbar_init(&drain_bar, 1);
        s_abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        if (FORM == DL) prefetch_tensormap(&tmOut);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&s_tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    const Walk<FORM> w(a);
    constexpr int PASSES = SPLIT ? SEGMENTS : 1;

    if (warp == 0 && lane == 0) {
        // ---------------------------------------------------------- TMA producer
        const int boxes_b = (a.bn + 63) / 64;
        const uint32_t bytes = A_BYTES + (MN_B ? boxes_b * 64 * BK * 2 : a.bn * BK * 2);
        int it = 0;
        bool go = true;
        for (int u = blockIdx.x; go && u < w.n_units; u += gridDim.x) {
            const Unit t = unit_at<FORM>(w, a, u);
            for (int j = 0; go && j < t.tiles; ++j) {
                const int n0 = t.n0 + j * a.bn;
                for (int c0 = t.k0; go && c0 < t.k1;) {
                    const int c1 = SPLIT && c0 + SPLIT_CHUNK < t.k1 ? c0 + SPLIT_CHUNK : t.k1;
                    for (int p = 0; go && p < PASSES; ++p) {
                        const int pa = SPLIT ? PLANE_A[p] : 0, pb = SPLIT ? PLANE_B[p] : 0;
                        for (int k = c0; k < c1; ++k, ++it) {
                            const int s = it % STAGES;
                            if (it >= STAGES)
                                go = wait_or_abort(&empty_bar[s], ((it / STAGES) - 1) & 1, &s_abort);
                            if (!go) break;
                            unsigned char *sa = smem + s * STAGE_BYTES, *sb = sa + A_BYTES;
                            mbar_arrive_expect_tx(&full_bar[s], bytes);
                            if (MN_A) {
                                for (int b = 0; b < BM / 64; ++b)
                                    tma_load_3d(sa + b * (64 * BK * 2), &tmA, &full_bar[s], t.m0 + b * 64,
                                                k * BK, pa);
                            } else {
                                tma_load_3d(sa, &tmA, &full_bar[s], k * BK, t.m0, pa);
                            }
                            if (MN_B) {
                                for (int b = 0; b < boxes_b; ++b)
                                    tma_load_3d(sb + b * (64 * BK * 2), &tmB, &full_bar[s], n0 + b * 64,
                                                (FORM == GX ? a.col0 : 0) + k * BK, pb);
                            } else {
                                tma_load_3d(sb, &tmB, &full_bar[s], k * BK, a.col0 + n0, pb);
                            }
                        }
                    }
                    c0 = c1;
                }
            }
        }
        if (!go)   // see the copies in flight through
            for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i)
                mbar_wait_bounded(&full_bar[i % STAGES], (i / STAGES) & 1, WAIT_NS, &g_vocab_error);
    } else if (warp == 1 && lane == 0) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc = idesc_bf16(BM, MN_A, MN_B) | static_cast<uint32_t>(a.bn >> 3) << 17;
        int it = 0, phase = 0;
        bool go = true;
        for (int u = blockIdx.x; go && u < w.n_units; u += gridDim.x) {
            const Unit t = unit_at<FORM>(w, a, u);
            for (int j = 0; go && j < t.tiles; ++j) {
                for (int c0 = t.k0; go && c0 < t.k1; ++phase) {
                    const int c1 = SPLIT && c0 + SPLIT_CHUNK < t.k1 ? c0 + SPLIT_CHUNK : t.k1;
                    const int buf = phase & 1;
                    if (phase >= 2) go = wait_or_abort(&acce_bar[buf], ((phase >> 1) - 1) & 1, &s_abort);
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t d = tmem + buf * BN;
                    const int its = (c1 - c0) * PASSES;
                    for (int i = 0; go && i < its; ++i, ++it) {
                        const int s = it % STAGES;
                        go = wait_or_abort(&full_bar[s], (it / STAGES) & 1, &s_abort);
                        if (!go) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint32_t sa = smem_u32(smem + s * STAGE_BYTES), sb = sa + A_BYTES;
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk) {
                            // 16 elements of K: 32 bytes of a K-major row, or 16 128-byte lines
                            const uint64_t da = MN_A ? sw128_mn_desc(sa + kk * 2048, 64 * BK * 2)
                                                     : sw128_desc(sa + kk * 32);
                            const uint64_t db = MN_B ? sw128_mn_desc(sb + kk * 2048, 64 * BK * 2)
                                                     : sw128_desc(sb + kk * 32);
                            mma_f16(d, da, db, idesc, i > 0 || kk > 0 ? 1u : 0u);
                        }
                        mma_commit(&empty_bar[s]);
                    }
                    if (go) mma_commit(&accf_bar[buf]);
                    c0 = c1;
                }
            }
        }
        if (!go) {   // see the products in flight through
            mma_commit(&drain_bar);
            mbar_wait_bounded(&drain_bar, 0, WAIT_NS, &g_vocab_error);
        }
    } else if (warp >= 4) {
        // --------------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        const int kept = *a.kept;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        unsigned char *stage_out = smem + STAGES * STAGE_BYTES + quarter * 2 * BOX_BYTES;
        int nblk = 0, phase = 0;
        bool ok = true;   // false once a wait gave up: NaN from there on
        for (int u = blockIdx.x; u < w.n_units; u += gridDim.x) {
            const Unit t = unit_at<FORM>(w, a, u);
            const int m = t.m0 + quarter * 32 + lane;   // this thread's row of the product
            // LSE, DL: the row's constants
            int target = -1;
            float lse2 = 0.f, gl = 0.f;
            if ((FORM == LSE || FORM == DL) && m < kept) {
                target = a.row[m].y - a.col0;
                if (FORM == DL) {
                    const float2 g = a.grad[m];
                    lse2 = g.x;
                    gl = g.y;
                }
            }
            const float scale2 = a.scale * LOG2E;
            float mx = __int_as_float(0xff800000), sum = 0.f;   // LSE: running maximum and sum

            // 32 columns c .. c + 31 of the tile at n0, as fp32
            auto take = [&](int n0, int c, float (&v)[32]) {
                const int left = a.n_cols - n0 - c;   // valid columns
                if (FORM == LSE) {
                    if (left <= 0) return;
                    float cm = __int_as_float(0xff800000);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        v[e] = e < left ? v[e] * scale2 : __int_as_float(0xff800000);
                        cm = fmaxf(cm, v[e]);
                    }
                    const float up = fmaxf(mx, cm);
                    const float ref = up == __int_as_float(0xff800000) ? 0.f : up;
                    float s = 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) s += ex2_approx(v[e] - ref);
                    sum = fmaf(sum, ex2_approx(mx - ref), s);
                    mx = up;
                    const int at = target - n0 - c;
                    if (at >= 0 && at < 32) {
                        float z = 0.f;
#pragma unroll
                        for (int e = 0; e < 32; ++e) z = e == at ? v[e] : z;
                        a.z_target[m] = z;
                    }
                } else if (FORM == DL) {
                    const int at = target - n0 - c;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float p = ex2_approx(fmaf(v[e], scale2, -lse2));
                        v[e] = m < kept && e < left ? gl * (e == at ? p - 1.f : p) : 0.f;
                        if (!ok) v[e] = __int_as_float(0x7fffffff);
                    }
#pragma unroll
                    for (int pl = 0; pl < (SPLIT ? 3 : 1); ++pl) {
                        unsigned char *blk = stage_out + (nblk & 1) * BOX_BYTES;
                        if (lane == 0) bulk_wait_read<1>();   // this block's previous store has read it
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint4 pk;
                            uint32_t *o = reinterpret_cast<uint32_t *>(&pk);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float &lo = v[q * 8 + 2 * e], &hi = v[q * 8 + 2 * e + 1];
                                const __nv_bfloat162 h2 = __floats2bfloat162_rn(lo, hi);
                                o[e] = *reinterpret_cast<const uint32_t *>(&h2);
                                if (SPLIT) {   // the next plane takes the rest
                                    lo -= __low2float(h2);
                                    hi -= __high2float(h2);
                                }
                            }
                            *reinterpret_cast<uint4 *>(blk + lane * 64 + 16 * (q ^ ((lane >> 1) & 3))) = pk;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_3d(&tmOut, blk, n0 + c, t.m0 + quarter * 32, pl);
                            bulk_commit();
                        }
                        ++nblk;
                    }
                } else {
                    if (!ok)
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __int_as_float(0x7fffffff);
                    const int n = min(left, a.bn - c);
                    if (n <= 0) return;
                    if (FORM == GX && a.acc != nullptr) {
                        if (m >= kept) return;
                        float *to = a.acc + t.split * a.acc_plane + static_cast<int64_t>(m) * a.acc_pitch + n0 + c;
                        if (a.acc_add) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (e < n) v[e] += to[e];
                        }
                        store_cols<float>(to, v, n, n % 4 == 0);
                    } else {
                        int64_t row;
                        if (FORM == GX) {
                            if (m >= kept) return;
                            row = a.row[m].x;
                        } else {
                            if (m >= a.M) return;
                            row = static_cast<int64_t>(a.col0) + m;
                        }
                        T *to = static_cast<T *>(a.out) + row * a.d + n0 + c;
                        const bool wide = a.d % (16 / sizeof(T)) == 0 &&
                                          (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
                        store_cols<T>(to, v, n, wide);
                    }
                }
            };

            for (int j = 0; j < t.tiles; ++j) {
                const int n0 = t.n0 + j * a.bn;
                if (SPLIT) {
                    float acc[SPLIT_BN];
#pragma unroll
                    for (int e = 0; e < SPLIT_BN; ++e) acc[e] = 0.f;
                    for (int c0 = t.k0; c0 < t.k1; c0 += SPLIT_CHUNK, ++phase) {
                        const int buf = phase & 1;
                        ok &= wait_or_abort(&accf_bar[buf], (phase >> 1) & 1, &s_abort);
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                        for (int c = 0; c < SPLIT_BN; c += 32) {
                            if (c < a.bn) {
                                uint32_t v[32];
                                tmem_ld_cols<32>(tmem + lane_base + buf * BN + c, v);
#pragma unroll
                                for (int e = 0; e < 32; ++e) acc[c + e] += __uint_as_float(v[e]);
                            }
                        }
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        mbar_arrive(&acce_bar[buf]);
                    }
#pragma unroll
                    for (int c = 0; c < SPLIT_BN; c += 32) {
                        if (c < a.bn) {
                            float v[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = acc[c + e];
                            take(n0, c, v);
                        }
                    }
                } else if (t.k0 < t.k1) {
                    const int buf = phase & 1;
                    ok &= wait_or_abort(&accf_bar[buf], (phase >> 1) & 1, &s_abort);
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
                    for (int c = 0; c < a.bn; c += 32) {
                        uint32_t r[32];
                        tmem_ld_cols<32>(tmem + lane_base + buf * BN + c, r);
                        float v[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
                        take(n0, c, v);
                    }
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    mbar_arrive(&acce_bar[buf]);
                    ++phase;
                } else {   // nothing to sum: zeros (no kept rows)
#pragma unroll 1
                    for (int c = 0; c < a.bn; c += 32) {
                        float v[32] = {};
                        take(n0, c, v);
                    }
                }
            }
            if (FORM == LSE && m < kept) {
                if (!ok) sum = __int_as_float(0x7fffffff);
                const int groups = (w.tiles_n + a.group - 1) / a.group;
                a.part[static_cast<int64_t>(m) * groups + u / w.tiles_m] = make_float2(mx, sum);
            }
        }
        if (FORM == DL && lane == 0) bulk_wait_all();   // the stores are done before the CTA exits
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 2) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// ------------------------------------------------------------------ the rows
// Numbers the rows whose target takes part, in order: row[m] = {row, target}.
// One CTA; each round takes 1024 x ROUND targets.
constexpr int KEPT_THREADS = 1024, ROUND = 4;

template <typename Id>
__global__ void __launch_bounds__(KEPT_THREADS)
    k_kept_rows(const void *targets, int n, int64_t V, int64_t ignore, int2 *row, int *kept) {
    __shared__ int warp_sum[KEPT_THREADS / 32];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int base = 0;
    for (int64_t r0 = 0; r0 < n; r0 += KEPT_THREADS * ROUND) {
        int64_t id[ROUND];
        int mine = 0;
        const int64_t i0 = r0 + static_cast<int64_t>(t) * ROUND;
#pragma unroll
        for (int e = 0; e < ROUND; ++e) {
            id[e] = i0 + e < n ? static_cast<int64_t>(static_cast<const Id *>(targets)[i0 + e]) : -1;
            if (i0 + e >= n || id[e] == ignore || id[e] < 0 || id[e] >= V) id[e] = -1;
            mine += id[e] >= 0;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL_MASK, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sum[w] = incl;
        __syncthreads();
        int lower = 0, all = 0;
        for (int v = 0; v < KEPT_THREADS / 32; ++v) {
            lower += v < w ? warp_sum[v] : 0;
            all += warp_sum[v];
        }
        int at = base + lower + incl - mine;
#pragma unroll
        for (int e = 0; e < ROUND; ++e)
            if (id[e] >= 0) row[at++] = make_int2(static_cast<int>(i0 + e), static_cast<int>(id[e]));
        base += all;
        __syncthreads();
    }
    if (t == 0) *kept = base;
}

// Copies the kept rows of x to (planes, rows_pad, pitch) bf16, zeros after them
// up to a multiple of 128 rows and beyond column d; with lse given, the rows'
// constants of the DL form.  Then, with gx given, clears the rows of gx that
// take no part (a target out of range gives NaN).
struct GatherArgs {
    const void *x;
    const int2 *row;
    const int *kept;
    __nv_bfloat16 *out;
    int64_t rows_pad;
    int d, pitch;
    const float *lse, *gl;
    float scale;
    float2 *grad;
    void *gx;
    const void *targets;
    int64_t V, ignore;
    int n;
};

template <typename T>
__device__ __forceinline__ void copy_row(const T *src, __nv_bfloat16 *dst, int64_t plane, int d,
                                         int pitch, int lane) {
    for (int c = lane * 2; c < pitch; c += 64) {
        float v0 = src != nullptr && c < d ? to_f32(src[c]) : 0.f;
        float v1 = src != nullptr && c + 1 < d ? to_f32(src[c + 1]) : 0.f;
#pragma unroll
        for (int p = 0; p < (sizeof(T) == 4 ? 3 : 1); ++p) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
            *reinterpret_cast<__nv_bfloat162 *>(dst + p * plane + c) = h;
            v0 -= __low2float(h);
            v1 -= __high2float(h);
        }
    }
}

template <typename T, typename Id>
__global__ void __launch_bounds__(256) k_gather_rows(const GatherArgs a) {
    const int lane = threadIdx.x & 31;
    const int kept = *a.kept;
    const int padded = (kept + BM - 1) / BM * BM;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t m = blockIdx.x * 8 + (threadIdx.x >> 5); m < a.rows_pad; m += warps) {
        if (m < padded) {
            const int src = m < kept ? a.row[m].x : -1;
            copy_row<T>(src >= 0 ? static_cast<const T *>(a.x) + static_cast<int64_t>(src) * a.d : nullptr,
                        a.out + m * a.pitch, a.rows_pad * a.pitch, a.d, a.pitch, lane);
            if (a.grad != nullptr && m < kept && lane == 0)
                a.grad[m] = make_float2(a.lse[src] * LOG2E, a.gl[src] * a.scale);
        }
        if (a.gx != nullptr && m < a.n) {
            const int64_t id = static_cast<int64_t>(static_cast<const Id *>(a.targets)[m]);
            if (id == a.ignore || id < 0 || id >= a.V) {
                const T fill = from_f32<T>(id == a.ignore ? 0.f : __int_as_float(0x7fffffff));
                for (int c = lane; c < a.d; c += 32) static_cast<T *>(a.gx)[m * a.d + c] = fill;
            }
        }
    }
}

// W as (planes, V, pitch) bf16
template <typename T>
__global__ void __launch_bounds__(256)
    k_planes(const T *W, __nv_bfloat16 *out, int64_t V, int d, int pitch) {
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t v = blockIdx.x * 8 + (threadIdx.x >> 5); v < V; v += warps)
        copy_row<T>(W + v * d, out + v * pitch, V * pitch, d, pitch, threadIdx.x & 31);
}

// Joins the row's partial maxima and sums; a warp per row.  Rows that take no
// part: zeros (a target out of range: NaN).
template <typename Id>
__global__ void __launch_bounds__(256)
    k_loss_join(const float2 *__restrict__ part, int groups, const float *__restrict__ z_target,
                const int2 *__restrict__ row, const int *__restrict__ kept, const void *targets, int n,
                int64_t V, int64_t ignore, float *__restrict__ loss, float *__restrict__ lse) {
    const int lane = threadIdx.x & 31;
    const int64_t m = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (m >= n) return;
    if (m < *kept) {
        const float2 *p = part + m * groups;
        float mx = __int_as_float(0xff800000), s = 0.f;
        for (int g = lane; g < groups; g += 32) {
            const float2 q = p[g];
            const float up = fmaxf(mx, q.x);
            const float ref = up == __int_as_float(0xff800000) ? 0.f : up;
            s = s * ex2_approx(mx - ref) + q.y * ex2_approx(q.x - ref);
            mx = up;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float om = __shfl_xor_sync(FULL_MASK, mx, o), os = __shfl_xor_sync(FULL_MASK, s, o);
            const float up = fmaxf(mx, om);
            const float ref = up == __int_as_float(0xff800000) ? 0.f : up;
            s = s * ex2_approx(mx - ref) + os * ex2_approx(om - ref);
            mx = up;
        }
        if (lane == 0) {
            const float l2 = mx + log2f(s);
            const int i = row[m].x;
            lse[i] = l2 * LN2;
            loss[i] = (l2 - z_target[m]) * LN2;
        }
    }
    const int64_t id = static_cast<int64_t>(static_cast<const Id *>(targets)[m]);
    if (lane == 0 && (id == ignore || id < 0 || id >= V)) {
        const float v = id == ignore ? 0.f : __int_as_float(0x7fffffff);
        lse[m] = v;
        loss[m] = v;
    }
}

// gx rows from the sums over pieces and splits
template <typename T>
__global__ void __launch_bounds__(256)
    k_gx_join(const float *__restrict__ acc, int splits, int64_t plane, int pitch,
              const int2 *__restrict__ row, const int *__restrict__ kept, T *__restrict__ gx, int d) {
    const int lane = threadIdx.x & 31;
    const int64_t m = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (m >= *kept) return;
    T *to = gx + static_cast<int64_t>(row[m].x) * d;
    for (int c = lane; c < d; c += 32) {
        float s = 0.f;
        for (int q = 0; q < splits; ++q) s += acc[q * plane + m * pitch + c];
        to[c] = from_f32<T>(s);
    }
}

// ---------------------------------------------------------------- host side
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The sizes a call works with, the same for the workspace query and the call.
struct Plan {
    int planes, pitch, d_bn, tile_v;
    int64_t rows_pad;
    bool copy_w;
    int64_t piece;        // backward: vocabulary rows of a piece
    int pieces, splits, group, groups;
    bool acc;
    size_t kept, row, x, w, part, z, grad, dl, accs, total;
};

// bytes the piece of G may take
constexpr int64_t PIECE_BYTES = 1ll << 30;

Plan plan_for(int64_t n, int64_t d, int64_t V, int dtype, bool w_aligned, bool backward) {
    Plan p{};
    const bool split = dtype == NRNN_F32;
    p.planes = split ? 3 : 1;
    p.pitch = static_cast<int>((d + 7) / 8 * 8);
    p.rows_pad = ceil_div(n, BM) * BM;
    p.copy_w = split || d % 8 != 0 || !w_aligned;
    const int most = split ? SPLIT_BN : BN;
    // columns of gx and gW in equal tiles
    p.d_bn = static_cast<int>(ceil_div(ceil_div(d, ceil_div(d, most)), 16) * 16);
    const int64_t tiles_m = ceil_div(n, BM);
    p.tile_v = most;
    const int64_t tiles_v = ceil_div(V, p.tile_v);
    // about eight units per CTA
    p.group = static_cast<int>(tiles_m * tiles_v / (SMS * 8));
    p.group = p.group < 1 ? 1 : p.group > 16 ? 16 : p.group;
    p.groups = static_cast<int>(ceil_div(tiles_v, p.group));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    p.kept = take(sizeof(int));
    p.row = take(sizeof(int2) * n);
    p.x = take(sizeof(__nv_bfloat16) * p.planes * p.rows_pad * p.pitch);
    p.w = take(p.copy_w ? sizeof(__nv_bfloat16) * p.planes * V * p.pitch : 0);
    if (!backward) {
        p.part = take(sizeof(float2) * n * p.groups);
        p.z = take(sizeof(float) * n);
    } else {
        p.grad = take(sizeof(float2) * n);
        const int64_t all = ceil_div(V, BN) * BN;
        p.piece = PIECE_BYTES / (2 * p.planes * p.rows_pad) / BN * BN;
        p.piece = p.piece < 2048 ? 2048 : p.piece;
        p.piece = p.piece > all ? all : p.piece;
        p.pieces = static_cast<int>(ceil_div(V, p.piece));
        // split gx's long inner dimension when its tiles do not fill the SMs
        const int64_t tiles = tiles_m * ceil_div(d, p.d_bn);
        p.splits = static_cast<int>(tiles >= SMS * 2 ? 1 : ceil_div(SMS * 2, tiles));
        const int64_t most_splits = p.piece / 512 > 0 ? p.piece / 512 : 1;
        p.splits = static_cast<int>(p.splits < most_splits ? p.splits : most_splits);
        p.acc = p.pieces > 1 || p.splits > 1;
        p.dl = take(sizeof(__nv_bfloat16) * p.planes * p.rows_pad * p.piece);
        p.accs = take(p.acc ? sizeof(float) * p.splits * p.rows_pad * p.pitch : 0);
    }
    p.total = at;
    return p;
}

template <int FORM, typename T>
cudaError_t gemm(const CUtensorMap &tmA, const CUtensorMap &tmB, const CUtensorMap &tmOut,
                 const GemmArgs &a, int64_t most_units, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};
    static int sms_of[64];
    cudaError_t e = once_per_device(configured, [](int dev) {
        cudaError_t r = cudaFuncSetAttribute(k_vocab_gemm<FORM, T>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(GEMM_SMEM));
        int n = 0;
        if (r == cudaSuccess) r = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (r == cudaSuccess && dev < 64) sms_of[dev] = n;
        return r;
    });
    if (e != cudaSuccess) return e;
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    if (most_units > INT32_MAX) return cudaErrorInvalidConfiguration;
    const int64_t grid = most_units < sms_of[dev] ? most_units : sms_of[dev];
    k_vocab_gemm<FORM, T><<<static_cast<unsigned>(grid), GEMM_THREADS, GEMM_SMEM, s>>>(tmA, tmB, tmOut, a);
    return cudaGetLastError();
}

struct Call {
    const void *x, *W, *targets;
    int dtype, targets_type;
    int64_t n, d, V, ignore;
    float scale;
    unsigned char *ws;
    cudaStream_t stream;
};

// kept rows, their copy, and W's planes if it needs any; returns W as bf16 planes
template <typename T, typename Id>
cudaError_t lay_out(const Call &c, const Plan &p, const float *lse, const float *gl, void *gx,
                    const void **w_out) {
    int *kept = reinterpret_cast<int *>(c.ws + p.kept);
    int2 *row = reinterpret_cast<int2 *>(c.ws + p.row);
    k_kept_rows<Id><<<1, KEPT_THREADS, 0, c.stream>>>(c.targets, static_cast<int>(c.n), c.V, c.ignore,
                                                      row, kept);
    GatherArgs g{};
    g.x = c.x; g.row = row; g.kept = kept;
    g.out = reinterpret_cast<__nv_bfloat16 *>(c.ws + p.x);
    g.rows_pad = p.rows_pad; g.d = static_cast<int>(c.d); g.pitch = p.pitch;
    g.lse = lse; g.gl = gl; g.scale = c.scale;
    g.grad = lse != nullptr ? reinterpret_cast<float2 *>(c.ws + p.grad) : nullptr;
    g.gx = gx; g.targets = c.targets; g.V = c.V; g.ignore = c.ignore; g.n = static_cast<int>(c.n);
    const int64_t blocks = p.rows_pad / 8;
    k_gather_rows<T, Id><<<static_cast<unsigned>(blocks < 4864 ? blocks : 4864), 256, 0, c.stream>>>(g);
    *w_out = c.W;
    if (p.copy_w) {
        __nv_bfloat16 *w = reinterpret_cast<__nv_bfloat16 *>(c.ws + p.w);
        const int64_t b = ceil_div(c.V, 8);
        k_planes<T><<<static_cast<unsigned>(b < 4864 ? b : 4864), 256, 0, c.stream>>>(
            static_cast<const T *>(c.W), w, c.V, static_cast<int>(c.d), p.pitch);
        *w_out = w;
    }
    return cudaGetLastError();
}

template <typename T, typename Id>
int forward(const Call &c, float *loss, float *lse) {
    const Plan p = plan_for(c.n, c.d, c.V, c.dtype, reinterpret_cast<uintptr_t>(c.W) % 16 == 0, false);
    const void *w;
    if (lay_out<T, Id>(c, p, nullptr, nullptr, nullptr, &w) != cudaSuccess) return NRNN_ERR_CUDA;
    CUtensorMap tmA, tmB;
    if (!make_map_planes(&tmA, c.ws + p.x, p.pitch, p.rows_pad, p.planes, BK, BM, true) ||
        !make_map_planes(&tmB, w, p.pitch, c.V, p.planes, BK, p.tile_v, true))
        return NRNN_ERR_CUDA;
    GemmArgs a{};
    a.kept = reinterpret_cast<int *>(c.ws + p.kept);
    a.M = -1; a.K = static_cast<int>(c.d);
    a.bn = p.tile_v; a.n_cols = static_cast<int>(c.V);
    a.group = p.group;
    a.scale = c.scale;
    a.row = reinterpret_cast<int2 *>(c.ws + p.row);
    a.part = reinterpret_cast<float2 *>(c.ws + p.part);
    a.z_target = reinterpret_cast<float *>(c.ws + p.z);
    if (gemm<LSE, T>(tmA, tmB, tmA, a, ceil_div(c.n, BM) * p.groups, c.stream) != cudaSuccess)
        return NRNN_ERR_CUDA;
    k_loss_join<Id><<<static_cast<unsigned>(ceil_div(c.n, 8)), 256, 0, c.stream>>>(
        a.part, p.groups, a.z_target, a.row, a.kept, c.targets, static_cast<int>(c.n), c.V, c.ignore,
        loss, lse);
    return cudaGetLastError() == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

template <typename T, typename Id>
int backward(const Call &c, const float *lse, const float *gl, void *gx, void *gW) {
    const Plan p = plan_for(c.n, c.d, c.V, c.dtype, reinterpret_cast<uintptr_t>(c.W) % 16 == 0, true);
    const void *w;
    if (lay_out<T, Id>(c, p, lse, gl, gx, &w) != cudaSuccess) return NRNN_ERR_CUDA;
    unsigned char *x = c.ws + p.x, *dl = c.ws + p.dl;
    CUtensorMap xk, wk, gk, wn, gn, xn, gs;   // K-major x, W, G; MN-major W, G, x; G's stores
    const int tile_v = p.tile_v;
    if (!make_map_planes(&xk, x, p.pitch, p.rows_pad, p.planes, BK, BM, true) ||
        !make_map_planes(&wk, w, p.pitch, c.V, p.planes, BK, tile_v, true) ||
        !make_map_planes(&gk, dl, p.piece, p.rows_pad, p.planes, BK, BM, true) ||
        !make_map_planes(&wn, w, p.pitch, c.V, p.planes, 64, BK, true) ||
        !make_map_planes(&gn, dl, p.piece, p.rows_pad, p.planes, 64, BK, true) ||
        !make_map_planes(&xn, x, p.pitch, p.rows_pad, p.planes, 64, BK, true) ||
        !make_map_planes(&gs, dl, p.piece, p.rows_pad, p.planes, BOX, BOX, false))
        return NRNN_ERR_CUDA;
    GemmArgs a{};
    a.kept = reinterpret_cast<int *>(c.ws + p.kept);
    a.scale = c.scale;
    a.row = reinterpret_cast<int2 *>(c.ws + p.row);
    a.grad = reinterpret_cast<float2 *>(c.ws + p.grad);
    a.d = static_cast<int>(c.d);
    a.splits = p.splits;
    a.acc_plane = p.rows_pad * p.pitch;
    a.acc_pitch = p.pitch;
    const int64_t tiles_m = ceil_div(c.n, BM), tiles_d = ceil_div(c.d, p.d_bn);
    for (int i = 0; i < p.pieces; ++i) {
        const int64_t v0 = i * p.piece;
        const int cols = static_cast<int>(c.V - v0 < p.piece ? c.V - v0 : p.piece);
        a.col0 = static_cast<int>(v0);
        a.M = -1; a.K = static_cast<int>(c.d);
        a.bn = tile_v; a.n_cols = cols;
        if (gemm<DL, T>(xk, wk, gs, a, tiles_m * ceil_div(cols, tile_v), c.stream) != cudaSuccess)
            return NRNN_ERR_CUDA;
        a.bn = p.d_bn; a.n_cols = a.d;
        a.K = cols;
        a.out = gx;
        a.acc = p.acc ? reinterpret_cast<float *>(c.ws + p.accs) : nullptr;
        a.acc_add = i > 0;
        if (gemm<GX, T>(gk, wn, gs, a, tiles_m * tiles_d * p.splits, c.stream) != cudaSuccess)
            return NRNN_ERR_CUDA;
        a.M = cols; a.K = -1;
        a.out = gW;
        a.acc = nullptr;
        if (gemm<GW, T>(gn, xn, gs, a, ceil_div(cols, BM) * tiles_d, c.stream) != cudaSuccess)
            return NRNN_ERR_CUDA;
    }
    if (p.acc)
        k_gx_join<T><<<static_cast<unsigned>(ceil_div(c.n, 8)), 256, 0, c.stream>>>(
            reinterpret_cast<float *>(c.ws + p.accs), p.splits, a.acc_plane, p.pitch, a.row, a.kept,
            static_cast<T *>(gx), a.d);
    return cudaGetLastError() == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

int check_vocab(const Call &c) {
    if (c.dtype != NRNN_F32 && c.dtype != NRNN_BF16) return NRNN_ERR_INVALID_ARG;
    if (c.targets_type != NRNN_I32 && c.targets_type != NRNN_I64) return NRNN_ERR_INVALID_ARG;
    if (c.n < 0 || c.d <= 0 || c.V <= 0) return NRNN_ERR_INVALID_ARG;
    if (c.n > (1 << 30) || c.d > (1 << 20) || c.V > (1 << 30)) return NRNN_ERR_UNSUPPORTED;
    const size_t elem = c.dtype == NRNN_BF16 ? 2 : 4, id = c.targets_type == NRNN_I64 ? 8 : 4;
    if (c.W == nullptr || (c.n > 0 && (c.x == nullptr || c.targets == nullptr))) return NRNN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(c.x) | reinterpret_cast<uintptr_t>(c.W)) % elem != 0 ||
        reinterpret_cast<uintptr_t>(c.targets) % id != 0)
        return NRNN_ERR_INVALID_ARG;
    return NRNN_OK;
}

}  // namespace
}  // namespace nrnn

using namespace nrnn;

extern "C" {

size_t nrnn_vocab_loss_workspace_bytes(int64_t rows, int64_t d, int64_t V, int dtype, int backward) {
    if (rows < 0 || d <= 0 || V <= 0 || rows > (1 << 30) || d > (1 << 20) || V > (1 << 30) ||
        (dtype != NRNN_F32 && dtype != NRNN_BF16))
        return 0;
    return plan_for(rows, d, V, dtype, false, backward != 0).total;
}

int nrnn_vocab_loss_forward(const void *x, const void *W, int dtype, int64_t rows, int64_t d,
                            int64_t V, const void *targets, int targets_type, int64_t ignore_index,
                            float logit_scale, float *loss, float *lse, void *workspace,
                            size_t ws_bytes, void *stream) {
    const Call c{x, W, targets, dtype, targets_type, rows, d, V, ignore_index, logit_scale,
                 static_cast<unsigned char *>(workspace), static_cast<cudaStream_t>(stream)};
    const int st = check_vocab(c);
    if (st != NRNN_OK) return st;
    if (rows == 0) return NRNN_OK;
    if (loss == nullptr || lse == nullptr) return NRNN_ERR_INVALID_ARG;
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
        ws_bytes < plan_for(rows, d, V, dtype, reinterpret_cast<uintptr_t>(W) % 16 == 0, false).total)
        return NRNN_ERR_WORKSPACE;
    const bool i64 = targets_type == NRNN_I64;
    if (dtype == NRNN_BF16)
        return i64 ? forward<__nv_bfloat16, int64_t>(c, loss, lse) : forward<__nv_bfloat16, int32_t>(c, loss, lse);
    return i64 ? forward<float, int64_t>(c, loss, lse) : forward<float, int32_t>(c, loss, lse);
}

int nrnn_vocab_loss_backward(const void *x, const void *W, int dtype, int64_t rows, int64_t d,
                             int64_t V, const void *targets, int targets_type, int64_t ignore_index,
                             float logit_scale, const float *lse, const float *g_loss, void *gx,
                             void *gW, void *workspace, size_t ws_bytes, void *stream) {
    const Call c{x, W, targets, dtype, targets_type, rows, d, V, ignore_index, logit_scale,
                 static_cast<unsigned char *>(workspace), static_cast<cudaStream_t>(stream)};
    const int st = check_vocab(c);
    if (st != NRNN_OK) return st;
    const size_t elem = dtype == NRNN_BF16 ? 2 : 4;
    if (gW == nullptr || (rows > 0 && (lse == nullptr || g_loss == nullptr || gx == nullptr)))
        return NRNN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(gx) | reinterpret_cast<uintptr_t>(gW)) % elem != 0)
        return NRNN_ERR_INVALID_ARG;
    if (rows == 0)
        return cudaMemsetAsync(gW, 0, elem * V * d, c.stream) == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
        ws_bytes < plan_for(rows, d, V, dtype, reinterpret_cast<uintptr_t>(W) % 16 == 0, true).total)
        return NRNN_ERR_WORKSPACE;
    const bool i64 = targets_type == NRNN_I64;
    if (dtype == NRNN_BF16)
        return i64 ? backward<__nv_bfloat16, int64_t>(c, lse, g_loss, gx, gW)
                   : backward<__nv_bfloat16, int32_t>(c, lse, g_loss, gx, gW);
    return i64 ? backward<float, int64_t>(c, lse, g_loss, gx, gW)
               : backward<float, int32_t>(c, lse, g_loss, gx, gW);
}

}  // extern "C"
