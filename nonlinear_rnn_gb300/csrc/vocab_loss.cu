// Softmax cross entropy over a vocabulary without keeping the logits, and its
// gradient in pieces of the vocabulary.
//
//   z_iv = c <x_i, W_v>,  lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_i,t(i)
//   G_iv = gl_i c (exp(z_iv - lse_i) - [v = t(i)]),  gx = G W,  gW = G^T x
//
// 2 N V d operations forward, 6 N V d backward (the logits are computed again):
// bound by the tensor cores, except for few rows, where reading W bounds it.
//
// All three products run on one persistent tcgen05 kernel (k_vocab_gemm): a pair
// of CTAs on two SMs (cta_group::2) per 256 x (up to 256) tile, TMA into a ring of
// 128-byte-swizzled stages, one thread issuing tcgen05.mma into one of two TMEM
// accumulators while the epilogue warps drain the other.  Each CTA of a pair stages
// half of B for both: the same tensor activity as one CTA per 128 x 256 tile (77% at
// 1.9 GHz), but 5% faster where the power limit sets the clock.  The kernel's forms
// differ in the operands' orientation (the transposed ones are read MN-major from
// where they lie: no transposed copy is made) and in the epilogue:
//   LSE  x W^T   running maximum and sum of each row over the unit's vocabulary
//   DL   x W^T   G of one piece of the vocabulary, to the workspace
//   GX   G W     gx, or this piece's share of it
//   GW   G^T x   rows of gW of this piece
// G of a piece, up to 1 GiB, is all that is ever kept of an N x V matrix (all of it where
// it fits).
//
// GX and GW have few output tiles and long inner dimensions.  Whole waves of tiles
// go one to a pair, which walk the inner dimension side by side and share what they
// read in L2, the column tiles of one row tile to a team of pairs beside one
// another; the tiles that do not fill a wave are cut by inner slices, an equal run
// of the (row tile, slice) sequence to every team.  A tile that is cut leaves fp32
// parts in the workspace, which k_join_parts adds in order.  (Whole tiles only: gx
// of 16384 x 1024 was 512 tiles on 152 SMs, 84% of them busy on average.  All tiles
// by slices: the CTAs read G at different places, and slower.)
//
// Rows whose target is ignored take no part: the kept rows are numbered on the
// device and gathered (k_kept_rows, k_gather_rows), and the kernel reads their
// number there, so ignored rows cost nothing and whatever they hold (infinities,
// NaN) reaches no output.
//
// For bf16 inputs G is rounded to bf16: both operands of a product have to be of one
// type, fp16 has not the range, and a second plane of G would make six products of the
// four (forward included).  The results are rounded to bf16 too and are off by that alone nearly as much
// (1.04 to 1.2 times it, 1.45 at most; see mantissa_of and TWO_PLANES_MOST).
//
// fp32 inputs are written as three bf16 planes, v = hi + mid + lo up to 2^-24 (values
// below 2^-110 less exactly: their lower planes are subnormal), and a
// product is the six plane products above 2^-24 relative, smallest first:
// (lo,hi) (mid,mid) (hi,lo) (mid,hi) (hi,mid) (hi,hi).  (An infinity leaves
// no number, so in W or in a kept row it counts as NaN.)  The tensor cores add less
// exactly than fp32 rounding does: every step of 16 drops what lies below the running
// sum's last bit (bf16 logits of 1024 products: lse 3e-7 off, fp32 products 4e-8).  So
// an accumulator takes at most 256 elements of the inner dimension before the epilogue
// adds it to fp32 registers.  (3001 rows over 10007 x 250: 512 elements gx 8.0e-7 off,
// 256 4.5e-7 in the same time, 128 2.7e-7 in 2% more; fp32 products 7.6e-7.)
//
// Measured: 16384 rows over 65536 x 1024 bf16 with gradient 5.2 to 5.6 ms (1.56 to
// 1.68 PFLOP/s; cuBLAS runs at 1.75 when kept up: the power limit holds the clocks at
// 1.7 GHz); 4096 over 32768 x 512 bf16 0.42 ms (1.2 PFLOP/s: a tile's 8 slices hide
// less of its epilogue), 3001 over 10007 x 250 fp32 0.292 ms, 4 rows over 50021 x 1024
// bf16, forward only, 31 to 37 us (W once in 20 to 23 us).  Without its epilogue the forward's
// main loop takes 0.96 of the time at d = 1024, 0.94 at 512 and 0.55 at 64, where the
// exponentials bind.
//
// Every wait is bounded.  One that gives up sets the call's error word (the
// workspace's second) and the abort flag of both CTAs of the pair, which ends the
// other roles' waits too: the producers and the issuer stop, and the epilogues hand
// back no accumulator and write NaN from there on.  Neither CTA leaves before the
// copies and products that both have in flight are done (settle).
#include "../../include/nrnn.h"
#include "nrnn_device.cuh"
#include "nrnn_internal.h"
#include "pair.cuh"
#include "rows.cuh"

namespace nrnn {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int PAIRS = 76;   // of 152 SMs: the work is divided for this many

enum Form { LSE, DL, GX, GW };

// GX, GW: the column tiles of a row tile go to as many pairs beside one another, up
// to this many
constexpr int MOST_SIDE = 8;

constexpr int BM = 256, BN = 256, BK = 64, STAGES = 6;   // of a pair
constexpr int HALF_M = BM / 2;                             // rows of A and D in one CTA
constexpr int A_BYTES = HALF_M * BK * 2, B_BYTES = BN / 2 * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8;   // two per 32 TMEM lanes: one alone on its scheduler waits on its own results
constexpr int GEMM_THREADS = 128 + EPI_WARPS * 32;
constexpr int PIECE = 64;                                  // columns that an epilogue warp takes at a time
constexpr int BOX_ROWS = 32, BOX_BYTES = BOX_ROWS * PIECE * 2;   // a stored block of G
constexpr size_t GEMM_SMEM = STAGES * STAGE_BYTES + EPI_WARPS * BOX_BYTES + 1024;
constexpr int SPLIT_CHUNK = 4;     // fp32: 64-wide slices per accumulator
constexpr int SEGMENTS = 6;        // fp32: plane products, smallest first
__device__ constexpr int PLANE_A[SEGMENTS] = {2, 1, 0, 1, 0, 0};
__device__ constexpr int PLANE_B[SEGMENTS] = {0, 1, 2, 0, 1, 0};

struct GemmArgs {
    const int *kept;          // device: number of kept rows
    uint32_t *error;          // device: set by a wait that gave up
    uint64_t wait_ns;         // limit of a wait
    int M;                    // rows of the product on the host's side: -1 = kept
    int K;                    // inner size: -1 = kept
    int bn;                   // columns of a tile: a multiple of 32, at most BN
    int a_rows;               // LSE, DL: rows of x that rank 0 reads (a multiple of 8); below
                              // HALF_M rank 1 reads none: rows past the last one are not used
    int n_cols;               // columns of the product (LSE, DL: of this piece)
    int col0;                 // LSE, DL: first vocabulary row; GX: B's first inner row;
                              // GW: first row of gW
    int group;                // LSE: column tiles a unit takes one after another
    float *parts;             // GX, GW: [pairs][2][BM][bn] sums of cut tiles
    float scale;              // logit scale c
    const int2 *row;          // per kept row {its row in x, its target}
    const float4 *grad;       // DL: per kept row, see row_grad
    const float *back;        // GX, GW of bf16: what G was divided by
    int g_planes;             // bf16: planes of G, 1 or 2
    float2 *part;             // LSE: [rows][groups][2] {maximum, sum} in base 2
    float *z_target;          // LSE: the target's product <x, W_t>
    void *out;                // GX, GW: the gradient in the storage type
    float *acc;               // GX: [rows][acc_pitch] sums over the pieces, if there are several
    int acc_pitch;
    bool acc_in, acc_out;     // GX: add acc; store to acc instead of out
    int d;                    // width of gx and gW rows
    bool blocks_out;          // GW: tmOut is over gW, whose blocks leave by TMA as whole lines (4
                              // rows over 50021 x 1024 bf16 with gradient: 139 -> 121 us)
};

template <typename T> __device__ __forceinline__ void store_cols(T *p, const float (&v)[PIECE], int n, bool wide) {
    constexpr int VEC = 16 / sizeof(T);
    if (wide) {
#pragma unroll
        for (int c = 0; c < PIECE; c += VEC) {
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = v[c + e];
            if (c < n) store_f32<T, VEC>(p + c, o);
        }
    } else {
#pragma unroll
        for (int c = 0; c < PIECE; ++c)
            if (c < n) p[c] = from_f32<T>(v[c]);
    }
}

__device__ __forceinline__ void times(float (&v)[PIECE], float f) {
    float2 *p = reinterpret_cast<float2 *>(v);
#pragma unroll
    for (int e = 0; e < PIECE / 2; ++e) p[e] = mul2(p[e], make_float2(f, f));
}

// A unit is what a pair takes at a time: a tile; `group` tiles beside one another
// (LSE); or a tile's slices k0 .. k1 (GX, GW).  Every role walks the same sequence.
struct Unit { int m0, n0, tiles, k0, k1, group, slot; };   // slot: -1 = a whole tile

template <int FORM> struct Walk {
    int tiles_m, tiles_n, n_units, kb, u;   // kb: 64-wide slices of the inner dimension
    int whole;                              // GX, GW: tiles that are not cut
    int64_t pos, end;                       // this team's run of (row tile - whole, slice)
    int pairs, side, side_at, teams;

    __device__ Walk(const GemmArgs &a, int pair, int pairs_) : pairs(pairs_) {
        const int kept = *a.kept;
        const int M = a.M < 0 ? kept : a.M, K = a.K < 0 ? kept : a.K;
        tiles_m = (M + BM - 1) / BM;
        tiles_n = (a.n_cols + a.bn - 1) / a.bn;
        kb = (K + BK - 1) / BK;
        n_units = tiles_m * (FORM == LSE ? (tiles_n + a.group - 1) / a.group : tiles_n);
        u = pair;
        if (FORM == LSE || FORM == DL) return;
        // teams of pairs with the column tiles of one row tile side by side
        side = tiles_n <= MOST_SIDE && tiles_n <= pairs ? tiles_n : 1;
        teams = pairs / side;
        side_at = pair % side;
        n_units /= side;
        whole = kb == 0 ? n_units : n_units / teams * teams;   // nothing to sum: zeros, tile by tile
        u = pair / side;
        if (u < teams) {
            run(u, pos, end);
        } else {   // a pair left over
            u = n_units;
            pos = end = 0;
        }
    }
    // the run of team b
    __device__ void run(int b, int64_t &from, int64_t &to) const {
        const int64_t all = static_cast<int64_t>(n_units - whole) * kb;
        from = all * b / teams;
        to = all * (b + 1) / teams;
    }
    __device__ __forceinline__ bool next(const GemmArgs &a, Unit &t) {
        t.k0 = 0; t.k1 = kb; t.tiles = 1; t.group = 0; t.slot = -1;
        if (FORM == LSE || FORM == DL) {
            if (u >= n_units) return false;
            // rows fastest: the pairs working at one time share a tile of W
            t.m0 = u % tiles_m * BM;
            t.group = u / tiles_m;
            t.n0 = t.group;
            if (FORM == LSE) {
                t.n0 *= a.group;
                t.tiles = tiles_n - t.n0 < a.group ? tiles_n - t.n0 : a.group;
            }
            t.n0 *= a.bn;
            u += pairs;
            return true;
        }
        int tile = u;
        if (u < whole) {
            u += teams;
        } else {
            if (pos >= end) return false;
            tile = whole + static_cast<int>(pos / kb);
            t.k0 = static_cast<int>(pos % kb);
            if (end - pos < kb - t.k0) t.k1 = t.k0 + static_cast<int>(end - pos);
            pos += t.k1 - t.k0;
            if (t.k0 > 0) t.slot = 0;
            else if (t.k1 < kb) t.slot = 1;
        }
        t.n0 = (side > 1 ? side_at : tile % tiles_n) * a.bn;
        t.m0 = (side > 1 ? tile : tile / tiles_n) * BM;
        return true;
    }
};

// PIECE (or fewer: n) columns from c of row m of the GX or GW product to their place
template <int FORM, typename T>
__device__ __forceinline__ void store_product(const GemmArgs &a, int kept, float back, int m, int c, float (&v)[PIECE],
                                              int n) {
    int64_t row;
    if (FORM == GX) {
        if (m >= kept) return;
        if (a.acc_in || a.acc_out) {
            float *to = a.acc + static_cast<int64_t>(m) * a.acc_pitch + c;
            if (a.acc_in) {
#pragma unroll
                for (int e = 0; e < PIECE; ++e)
                    if (e < n) v[e] += to[e];
            }
            if (a.acc_out) {
                store_cols<float>(to, v, n, n % 4 == 0);
                return;
            }
        }
        row = a.row[m].x;
    } else {
        if (m >= a.M) return;
        row = static_cast<int64_t>(a.col0) + m;
    }
    if (sizeof(T) == 2) times(v, back);
    const bool wide = a.d % (16 / sizeof(T)) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
    store_cols<T>(static_cast<T *>(a.out) + row * a.d + c, v, n, wide);
}

// rows of x below one CTA's: rank 1 reads none
template <int FORM> __device__ __forceinline__ bool few_rows_of_a(const GemmArgs &a) {
    return (FORM == LSE || FORM == DL) && a.a_rows < HALF_M;
}
// bytes of a stage's copies in the CTA of a rank: one box of a K-major operand, 64
// columns each of an MN-major one
template <int FORM> __device__ __forceinline__ uint32_t stage_bytes(const GemmArgs &a, int rank) {
    const int half_n = a.bn / 2, b_rows = FORM == GX || FORM == GW ? (half_n + 63) / 64 * 64 : half_n;
    return (!few_rows_of_a<FORM>(a) ? A_BYTES : rank == 0 ? a.a_rows * BK * 2 : 0) + b_rows * BK * 2;
}

// T: storage type of the inputs (float: split products)
template <int FORM, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GEMM_THREADS, 1)
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
    __shared__ volatile uint32_t s_abort;     // a role of either CTA gave up
    __shared__ volatile int s_issued[2];      // rank 0's: stages that each producer went through

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);   // rank 0's: both CTAs' copies
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 1);
            mbar_init(&acce_bar[b], 2 * EPI_WARPS);   // rank 0's: both epilogues
        }
        mbar_init(&drain_bar, 1);
        s_abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        if (FORM == DL || FORM == GW) prefetch_tensormap(&tmOut);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&s_tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync_all();   // both CTAs' barriers are there
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    dependents_may_launch();
    wait_for_prerequisites();
    const int pair = blockIdx.x >> 1;
    Walk<FORM> w(a, pair, gridDim.x >> 1);
    Unit t;
    constexpr int PASSES = SPLIT ? SEGMENTS : 1;
    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        // Lane i starts the i-th copy of a stage.  (One lane after another took longer than
        // the products of a stage: gW of 16384 x 65536 x 1024 ran at 1.4 PFLOP/s.)
        constexpr int BOXES_A = MN_A ? HALF_M / 64 : 1;
        const int half_n = a.bn / 2;
        const int boxes_b = MN_B ? (half_n + 63) / 64 : 1;
        const bool few = few_rows_of_a<FORM>(a);
        const uint32_t bytes = stage_bytes<FORM>(a, 0) + stage_bytes<FORM>(a, 1);
        const bool is_a = lane < BOXES_A;
        const bool copies = is_a ? rank == 0 || !few : lane < BOXES_A + boxes_b;
        const int box = is_a ? lane : lane - BOXES_A;
        const int twice = !SPLIT && (FORM == GX || FORM == GW) ? a.g_planes : 1;   // G's planes, smaller first
        const bool mn = is_a ? MN_A : MN_B;
        const uint32_t offset = (is_a ? 0 : A_BYTES) + box * (64 * BK * 2);
        int it = 0;
        bool go = true;
        while (go && w.next(a, t)) {
            for (int j = 0; go && j < t.tiles; ++j) {
                // this lane's coordinate along M or N
                const int at = is_a ? t.m0 + static_cast<int>(rank) * HALF_M + box * 64
                                    : (MN_B ? 0 : a.col0) + t.n0 + j * a.bn +
                                          static_cast<int>(rank) * half_n + box * 64;
                for (int c0 = t.k0; go && c0 < t.k1;) {
                    const int c1 = SPLIT && c0 + SPLIT_CHUNK < t.k1 ? c0 + SPLIT_CHUNK : t.k1;
                    for (int p = 0; go && p < PASSES; ++p) {
                        int plane = SPLIT ? (is_a ? PLANE_A[p] : PLANE_B[p]) : 0;
                        for (int i = 0; i < (c1 - c0) * twice; ++i, ++it) {
                            int k = c0 + i;
                            if (!SPLIT && twice == 2) {
                                k = c0 + (i >> 1);
                                plane = is_a ? 1 - (i & 1) : 0;
                            }
                            const int s = it % STAGES;
                            if (it >= STAGES)
                                go = __all_sync(FULL_MASK, wait_or_abort(a, &empty_bar[s], ((it / STAGES) - 1) & 1, &s_abort));
                            if (!go) break;
                            if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&full_bar[s], bytes);
                            __syncwarp();
                            const int along_k = k * BK + (FORM == GX && !is_a ? a.col0 : 0);
                            if (copies)
                                tma_load_3d_pair(smem + s * STAGE_BYTES + offset, is_a ? &tmA : &tmB,
                                                 cluster_addr(&full_bar[s], 0), mn ? at : along_k,
                                                 mn ? along_k : at, plane);
                        }
                    }
                    c0 = c1;
                }
            }
        }
        if (lane == 0) cluster_store(cluster_addr(const_cast<const int *>(&s_issued[rank]), 0), static_cast<uint32_t>(it));
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc = idesc_bf16(BM, MN_A, MN_B) | static_cast<uint32_t>(a.bn >> 3) << 17;
        int it = 0, phase = 0;
        bool go = true;
        while (go && w.next(a, t)) {
            for (int j = 0; go && j < t.tiles; ++j) {
                for (int c0 = t.k0; go && c0 < t.k1; ++phase) {
                    const int c1 = SPLIT && c0 + SPLIT_CHUNK < t.k1 ? c0 + SPLIT_CHUNK : t.k1;
                    const int buf = phase & 1;
                    if (phase >= 2) go = wait_or_abort(a, &acce_bar[buf], ((phase >> 1) - 1) & 1, &s_abort);
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t d = tmem + buf * BN;
                    const int its = (c1 - c0) * PASSES * (!SPLIT && (FORM == GX || FORM == GW) ? a.g_planes : 1);
                    for (int i = 0; go && i < its; ++i, ++it) {
                        const int s = it % STAGES;
                        go = wait_or_abort(a, &full_bar[s], (it / STAGES) & 1, &s_abort);
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
                            mma_f16_pair(d, da, db, idesc, i > 0 || kk > 0 ? 1u : 0u);
                        }
                        mma_commit_pair(&empty_bar[s]);
                    }
                    if (go) mma_commit_pair(&accf_bar[buf]);
                    c0 = c1;
                }
            }
        }
    } else if (warp >= 4) {
        // --------------------------------------------------------------- epilogue
        // warps 4..7 take the even pieces of their 32 rows, 8..11 the odd ones
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const int kept = *a.kept;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        unsigned char *stage_out = smem + STAGES * STAGE_BYTES + (warp - 4) * BOX_BYTES;
        const float scale2 = a.scale * LOG2E;
        constexpr float NEG_INF = -INFINITY;
        const float nan = __int_as_float(0x7fffffff);
        const float back = !SPLIT && (FORM == GX || FORM == GW) ? *a.back : 1.f;
        int phase = 0;
        bool ok = true;   // false once a wait gave up: NaN from there on
        auto release = [&](int buf) {   // this warp has read the accumulator
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive_cluster(cluster_addr(&acce_bar[buf], 0));
        };
        auto accumulator = [&](int buf, uint32_t parity) {
            ok &= wait_or_abort(a, &accf_bar[buf], parity, &s_abort);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        };
        while (w.next(a, t)) {
            const int in_tile = static_cast<int>(rank) * HALF_M + quarter * 32;   // the warp's first row
            const int m = t.m0 + in_tile + lane;   // this thread's row of the product
            // LSE, DL: the row's constants
            int target = -1;
            float lse2 = 0.f, gl = 0.f, gl_p = 0.f;
            if ((FORM == LSE || FORM == DL) && m < kept) {
                target = a.row[m].y - a.col0;
                if (FORM == DL) {
                    const float4 g = a.grad[m];
                    lse2 = g.x;
                    gl = g.y;
                    gl_p = g.z;
                }
            }
            // LSE: running maximum and sums.  Four chains each: one alone waits for
            // every step's result.
            float mx = NEG_INF;
            float2 sum[2] = {};

            // the warp's 32 x PIECE block, rounded to bf16, to column x and row y of tmOut;
            // with more planes than one, v keeps what rounding leaves for the next
            auto store_block = [&](float (&v)[PIECE], int x, int y, int plane, auto planes) {
                constexpr bool MORE = decltype(planes)::value > 1;
                if (lane == 0) bulk_wait_read<0>();   // the store before has read the block
                __syncwarp();
#pragma unroll
                for (int q = 0; q < PIECE / 8; ++q) {
                    uint4 pk;
                    uint32_t *o = reinterpret_cast<uint32_t *>(&pk);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &lo = v[q * 8 + 2 * e], &hi = v[q * 8 + 2 * e + 1];
                        const __nv_bfloat162 h2 =
                            MORE && plane == 0 ? finite_bf16x2(lo, hi) : __floats2bfloat162_rn(lo, hi);
                        o[e] = *reinterpret_cast<const uint32_t *>(&h2);
                        if (MORE) {
                            lo -= __low2float(h2);
                            hi -= __high2float(h2);
                        }
                    }
                    // 128-byte swizzle: 16-byte piece q of row r lies at q ^ (r & 7)
                    *reinterpret_cast<uint4 *>(stage_out + lane * 128 + 16 * (q ^ (lane & 7))) = pk;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&tmOut, stage_out, x, y, plane);
                    bulk_commit();
                }
            };

            // columns c .. c + PIECE - 1 of the tile at n0, as fp32
            auto take = [&](int n0, int c, float (&v)[PIECE]) {
                float2 *p = reinterpret_cast<float2 *>(v);
                const int left = min(a.n_cols - n0, a.bn) - c;   // valid columns
                if (left <= 0 && FORM != DL) return;
                if (FORM == LSE) {
                    // Sums of 2^(z scale2 - ref), the product not rounded by itself (as in DL, whose
                    // probabilities would not add up to one with this lse else, by 2.6e-6 at logits
                    // of 48).  The reference is the largest scaled logit, rounded, or near it.
                    const int at = target - n0 - c;
                    if (at >= 0 && at < min(left, PIECE)) {
                        float z = 0.f;
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) z = e == at ? v[e] : z;
                        a.z_target[m] = z;
                    }
                    if (scale2 < 0.f)
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) v[e] = -v[e];
                    const float s2 = fabsf(scale2);
                    if (left < PIECE)
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) v[e] = e < left ? v[e] : NEG_INF;
                    float up[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
                    for (int e = 0; e < PIECE; ++e) up[e % 4] = fmaxf(up[e % 4], v[e]);
                    const float most = fmaxf(mx, fmaxf(fmaxf(up[0], up[1]), fmaxf(up[2], up[3])) * s2);
                    const float ref = most == NEG_INF ? 0.f : most;
                    const float keep = ex2_approx(mx - ref);
                    mx = most;
#pragma unroll
                    for (int q = 0; q < 2; ++q) sum[q] = mul2(sum[q], make_float2(keep, keep));
                    if (left < PIECE) {   // what is outside adds nothing (also at a scale of zero)
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) {
                            const float x = e < left ? ex2_approx(fmaf(v[e], s2, -ref)) : 0.f;
                            (e % 2 == 0 ? sum[e / 2 % 2].x : sum[e / 2 % 2].y) += x;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < PIECE / 2; ++e) {
                            const float2 x = fma2(p[e], make_float2(s2, s2), make_float2(-ref, -ref));
                            sum[e % 2] = add2(sum[e % 2], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
                        }
                    }
                } else if (FORM == DL) {
#pragma unroll
                    for (int e = 0; e < PIECE / 2; ++e) {
                        const float2 x = fma2(p[e], make_float2(scale2, scale2), make_float2(-lse2, -lse2));
                        p[e] = mul2(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(gl_p, gl_p));
                    }
                    const int at = target - n0 - c;
                    if (at >= 0 && at < PIECE)
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) v[e] = e == at ? v[e] - gl : v[e];
                    if (left < PIECE || m >= kept)   // zeros outside, whatever the exponential gave
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) v[e] = e < left && m < kept ? v[e] : 0.f;
                    if (!ok)
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) v[e] = nan;
                    using std::integral_constant;
                    const int x = n0 + c, y = t.m0 + in_tile;
                    if (SPLIT) {
#pragma unroll
                        for (int pl = 0; pl < 3; ++pl) store_block(v, x, y, pl, integral_constant<int, 3>{});
                    } else if (a.g_planes == 2) {
#pragma unroll
                        for (int pl = 0; pl < 2; ++pl) store_block(v, x, y, pl, integral_constant<int, 2>{});
                    } else {
                        store_block(v, x, y, 0, integral_constant<int, 1>{});
                    }
                } else {
                    if (!ok)
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) v[e] = nan;
                    const int n = min(left, PIECE);
                    if (FORM == GW && !SPLIT && a.blocks_out && t.slot < 0) {
                        times(v, back);
                        if (t.m0 + in_tile < a.M)
                            store_block(v, n0 + c, a.col0 + t.m0 + in_tile, 0, std::integral_constant<int, 1>{});
                    } else if (t.slot < 0) {
                        store_product<FORM, T>(a, kept, back, m, n0 + c, v, n);
                    } else {
                        float *to = a.parts + ((static_cast<int64_t>(pair) * 2 + t.slot) * BM + in_tile + lane) * a.bn + c;
                        store_cols<float>(to, v, n, n % 4 == 0);
                    }
                }
            };

            for (int j = 0; j < t.tiles; ++j) {
                const int n0 = t.n0 + j * a.bn;
                if (SPLIT) {
                    constexpr int PIECES = BN / PIECE / 2;   // of this warp
                    float acc[PIECES][PIECE];
#pragma unroll
                    for (int i = 0; i < PIECES; ++i)
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) acc[i][e] = 0.f;
                    for (int c0 = t.k0; c0 < t.k1; c0 += SPLIT_CHUNK, ++phase) {
                        const int buf = phase & 1;
                        accumulator(buf, (phase >> 1) & 1);
#pragma unroll
                        for (int i = 0; i < PIECES; ++i)
#pragma unroll
                            for (int h = 0; h < PIECE; h += 32) {
                                const int c = (2 * i + half) * PIECE + h;
                                if (c < a.bn) {
                                    uint32_t v[32];
                                    tmem_ld_cols<32>(tmem + lane_base + buf * BN + c, v);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) acc[i][h + e] += __uint_as_float(v[e]);
                                }
                            }
                        release(buf);
                    }
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) {
                        const int c = (2 * i + half) * PIECE;
                        if (c < a.bn) take(n0, c, acc[i]);
                    }
                } else if (t.k0 < t.k1) {
                    const int buf = phase & 1;
                    accumulator(buf, (phase >> 1) & 1);
#pragma unroll 1
                    for (int c = half * PIECE; c < a.bn; c += 2 * PIECE) {
                        uint32_t r[PIECE];
                        tmem_ld_cols<PIECE>(tmem + lane_base + buf * BN + c, r);
                        float v[PIECE];
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) v[e] = __uint_as_float(r[e]);
                        if (c + 2 * PIECE >= a.bn) release(buf);   // the last piece is in registers
                        take(n0, c, v);
                    }
                    if (half * PIECE >= a.bn) release(buf);
                    ++phase;
                } else {   // nothing to sum: zeros (no kept rows)
#pragma unroll 1
                    for (int c = half * PIECE; c < a.bn; c += 2 * PIECE) {
                        float v[PIECE] = {};
                        take(n0, c, v);
                    }
                }
            }
            if (FORM == LSE && m < kept) {
                const int groups = (w.tiles_n + a.group - 1) / a.group;
                a.part[(static_cast<int64_t>(m) * groups + t.group) * 2 + half] =
                    make_float2(mx, ok ? (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y) : nan);
            }
        }
        if ((FORM == DL || FORM == GW) && lane == 0) bulk_wait_all();   // the stores are done before the CTA exits
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync_all();   // neither CTA leaves while the other may still reach into it
    if (s_abort != 0) {   // the same in both
        if (warp == 1 && lane == 0) {
            if (rank == 0) settle<STAGES>(a, s_issued, full_bar, &drain_bar, stage_bytes<FORM>(a, 1));
            else mbar_wait_bounded(&drain_bar, 0, SETTLE_NS, a.error);
        }
        __syncwarp();
        cluster_sync_all();
    }
    if (warp == 2) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// Adds the parts of the tiles that the GX or GW launch of `pairs` pairs cut, in the
// order of their slices.  blockIdx.x: a cut tile.  A warp takes a row, 8 columns a
// lane; with SPLIT_PARTS (few tiles in many parts) the CTA's warps take a share of
// one row's parts each, and the shares are added in order.
constexpr int JOIN_WARPS = 8;

template <int FORM, typename T, bool SPLIT_PARTS>
__global__ void __launch_bounds__(JOIN_WARPS * 32) k_join_parts(const GemmArgs a, int pairs) {
    __shared__ float share[SPLIT_PARTS ? JOIN_WARPS : 1][BN];
    dependents_may_launch();
    wait_for_prerequisites();
    const Walk<FORM> w(a, 0, pairs);
    const int cut = blockIdx.x / w.side, tile = w.whole + cut;   // among the row tiles of a team
    if (tile >= w.n_units) return;
    const int side_at = blockIdx.x % w.side;
    const int kept = *a.kept, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = SPLIT_PARTS ? blockIdx.y : blockIdx.y * JOIN_WARPS + warp;
    const int m = (w.side > 1 ? tile : tile / w.tiles_n) * BM + row;
    const int n0 = (w.side > 1 ? side_at : tile % w.tiles_n) * a.bn;
    if (m >= (FORM == GX ? kept : a.M)) return;
    // the runs that hold slices of this tile: b0 .. b1
    const int64_t all = static_cast<int64_t>(w.n_units - w.whole) * w.kb;
    const int64_t first = static_cast<int64_t>(cut) * w.kb, stop = first + w.kb;
    auto run_of = [&](int64_t slice) {   // the run that holds a slice
        int b = static_cast<int>(slice * w.teams / all);
        int64_t from, to;
        for (w.run(b, from, to); slice < from; w.run(--b, from, to)) {}
        for (; slice >= to; w.run(++b, from, to)) {}
        return b;
    };
    const int b0 = run_of(first), b1 = run_of(stop - 1);
    if (b0 == b1) return;   // one run has it whole
    const bool dense = all >= w.teams;   // no run is empty
    const int c = lane * 8;
    float v[8] = {};
    if (c < a.bn) {
        const int64_t step = static_cast<int64_t>(2) * BM * a.bn * w.side;   // to the next team's
        const float *p = a.parts + b0 * step + (static_cast<int64_t>(side_at) * 2 * BM + row) * a.bn + c;
        const int q0 = SPLIT_PARTS ? warp : 0, dq = SPLIT_PARTS ? JOIN_WARPS : 1;
#pragma unroll 4
        for (int q = q0; q <= b1 - b0; q += dq) {
            if (!dense) {
                int64_t f, t;
                w.run(b0 + q, f, t);
                if (f == t) continue;
            }
            // the first run's part begins with the tile: slot 1
            float x[8];
            load_f32<float, 8>(p + q * step + (q == 0 ? static_cast<int64_t>(BM) * a.bn : 0), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += x[e];
        }
    }
    if (SPLIT_PARTS) {
        if (c < a.bn)
#pragma unroll
            for (int e = 0; e < 8; ++e) share[warp][c + e] = v[e];
        __syncthreads();
        if (warp > 0 || c >= a.bn) return;
        for (int q = 1; q < JOIN_WARPS; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += share[q][c + e];
    }
    const int n = min(min(a.bn, a.n_cols - n0) - c, 8);
    if (n <= 0) return;
    const int col = n0 + c;
    int64_t at;
    if (FORM == GX) {
        float *acc = a.acc + static_cast<int64_t>(m) * a.acc_pitch + col;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (a.acc_in && e < n) v[e] += acc[e];
        if (a.acc_out) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) acc[e] = v[e];
            return;
        }
        at = static_cast<int64_t>(a.row[m].x) * a.d + col;
    } else {
        at = (static_cast<int64_t>(a.col0) + m) * a.d + col;
    }
    if (sizeof(T) == 2) {
        const float back = *a.back;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= back;
    }
    T *to = static_cast<T *>(a.out) + at;
    if (a.d % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0) {
#pragma unroll
        for (int e = 0; e < 8; e += 16 / sizeof(T)) {
            float o[16 / sizeof(T)];
#pragma unroll
            for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) o[i] = v[e + i];
            store_f32<T, 16 / sizeof(T)>(to + e, o);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) to[e] = from_f32<T>(v[e]);
    }
}

// ------------------------------------------------------------------ the rows
// Numbers the rows whose target takes part, in order: row[m] = {row, target}, by one
// CTA; each round takes THREADS x ROUND targets, 32 x ROUND consecutive ones a warp.
// Returns their number.
constexpr int KEPT_THREADS = 1024, GATHER_THREADS = 256, ROUND = 16;

template <int THREADS, typename Id>
__device__ __forceinline__ int number_rows(const void *targets, int n, int64_t V, int64_t ignore, int2 *row) {
    constexpr int WARPS = THREADS / 32;
    __shared__ int warp_sum[WARPS];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int base = 0;
    for (int64_t r0 = 0; r0 < n; r0 += THREADS * ROUND) {
        int64_t id[ROUND];
        unsigned vote[ROUND];
        int mine = 0;
        const int64_t i0 = r0 + w * (32 * ROUND) + lane;
#pragma unroll
        for (int e = 0; e < ROUND; ++e)
            id[e] = i0 + e * 32 < n ? static_cast<int64_t>(static_cast<const Id *>(targets)[i0 + e * 32]) : -1;
#pragma unroll
        for (int e = 0; e < ROUND; ++e) {
            vote[e] = __ballot_sync(FULL_MASK, i0 + e * 32 < n && id[e] != ignore && id[e] >= 0 && id[e] < V);
            mine += __popc(vote[e]);
        }
        if (lane == 0) warp_sum[w] = mine;
        __syncthreads();
        int all = lane < WARPS ? warp_sum[lane] : 0;
        int at = lane < w ? all : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            all += __shfl_xor_sync(FULL_MASK, all, o);
            at += __shfl_xor_sync(FULL_MASK, at, o);
        }
        at += base;
#pragma unroll
        for (int e = 0; e < ROUND; ++e) {
            if (vote[e] >> lane & 1u)
                row[at + __popc(vote[e] & ((1u << lane) - 1u))] =
                    make_int2(static_cast<int>(i0) + e * 32, static_cast<int>(id[e]));
            at += __popc(vote[e]);
        }
        base += all;
        __syncthreads();
    }
    return base;
}

template <typename Id>
__global__ void __launch_bounds__(KEPT_THREADS)
    k_kept_rows(const void *targets, int n, int64_t V, int64_t ignore, int2 *row, int *kept) {   // kept: {number, error}
    dependents_may_launch();
    wait_for_prerequisites();
    const int all = number_rows<KEPT_THREADS, Id>(targets, n, V, ignore, row);
    if (threadIdx.x == 0) kept[0] = all, kept[1] = 0;
}

// Copies the kept rows of x to (planes, rows_pad, pitch) bf16, zeros after them
// up to a multiple of 256 rows and beyond column d; with lse given, the rows'
// constants of the DL form.  Then, with gx given, clears the rows of gx that
// take no part (a target out of range gives NaN).  FEW: every CTA numbers the rows
// for itself (the first one for the kernels that follow too), which is sooner done
// than a launch before this one.
constexpr int FEW_ROWS = GATHER_THREADS * ROUND;

struct GatherArgs {
    const void *x;
    int2 *row;
    int *kept;
    __nv_bfloat16 *out;
    int64_t rows_pad;
    int d, pitch;
    const float *lse, *gl;
    float scale;
    float4 *grad;
    float *back;              // bf16: see mantissa_of
    void *gx;
    const void *targets;
    int64_t V, ignore;
    int n;
};

// The mantissa, in [1, 2), of a finite value that is not zero or subnormal; else 1.
// A bf16 G is divided by the mantissa of the first kept row's dL/dloss c, and its two
// products are multiplied by it at their end.  Where all rows have the same dL/dloss
// (a mean), their largest entries are then 1 - p times a power of two.  With the
// mantissa, entries of rows of small p would all be close to one value and be rounded
// alike: gx of 15 rows, G as one plane, is off by up to 2.05 times what rounding it
// costs with the mantissa and by 1.28 times without; of 1500 rows 1.47 and 1.14.
__device__ __forceinline__ float mantissa_of(float v) {
    const uint32_t bits = __float_as_uint(v), exponent = bits >> 23 & 0xffu;
    return exponent == 0 || exponent == 255 ? 1.f : __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
}

// A kept row's constants of the DL form: {l = lse log2(e), g, g 2^(l - lse log2(e))} with
// g = gl c / back.  What rounding l leaves out (2^-18 at an lse of 48) is put into the
// factor of p, which would be off by it.
__device__ __forceinline__ float4 row_grad(float lse, float g) {
    constexpr float LOG2E_LOW = 1.92596303e-8f;   // log2(e) less LOG2E
    const float l = lse * LOG2E, low = fmaf(lse, LOG2E, -l) + lse * LOG2E_LOW;
    return make_float4(l, g, isfinite(low) ? fmaf(-low * LN2, g, g) : g, 0.f);
}

template <typename T, typename Id, bool FEW>
__global__ void __launch_bounds__(GATHER_THREADS) k_gather_rows(const GatherArgs a) {
    __shared__ int2 few_rows[FEW ? FEW_ROWS : 1];
    dependents_may_launch();
    wait_for_prerequisites();
    const int lane = threadIdx.x & 31;
    const int2 *rows = a.row;
    int kept;
    if (FEW) {
        kept = number_rows<GATHER_THREADS, Id>(a.targets, a.n, a.V, a.ignore, few_rows);
        rows = few_rows;
        if (blockIdx.x == 0) {
            for (int i = threadIdx.x; i < kept; i += GATHER_THREADS) a.row[i] = few_rows[i];
            if (threadIdx.x == 0) a.kept[0] = kept, a.kept[1] = 0;
        }
    } else {
        kept = *a.kept;
    }
    const bool wide = wide_rows<T>(a.x, a.d);
    float back = 1.f;
    if (sizeof(T) == 2 && a.grad != nullptr) {
        if (kept > 0) back = mantissa_of(a.gl[rows[0].x] * a.scale);
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.back = back;
    }
    const int padded = (kept + BM - 1) / BM * BM;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t m = blockIdx.x * 8 + (threadIdx.x >> 5); m < a.rows_pad; m += warps) {
        if (m < padded) {
            const int src = m < kept ? rows[m].x : -1;
            copy_row<T>(src >= 0 ? static_cast<const T *>(a.x) + static_cast<int64_t>(src) * a.d : nullptr,
                        a.out + m * a.pitch, a.rows_pad * a.pitch, a.d, a.pitch, lane, wide);
            if (a.grad != nullptr && m < kept && lane == 0)
                a.grad[m] = row_grad(a.lse[src], a.gl[src] * a.scale / back);
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
    dependents_may_launch();
    wait_for_prerequisites();   // the planes' memory may still be read by the call before
    const bool wide = wide_rows<T>(W, d);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t v = blockIdx.x * 8 + (threadIdx.x >> 5); v < V; v += warps)
        copy_row<T>(W + v * d, out + v * pitch, V * pitch, d, pitch, threadIdx.x & 31, wide);
}

// ------------------------------------------------------------ few rows, fp32
// lse of at most FEW_MOST fp32 rows on the fp32 cores: writing W's planes and reading
// them back would be four times the bytes that W has (33 rows over 47579 x 552: 126
// us).  A warp takes FEW_V rows of W at a time, 128 bytes a lane apart, against every
// row of x from shared memory, so a value of x that is read serves FEW_V products.
// One row over 50021 x 1024 reads W at 0.70 of HBM (44 us), four at 0.58 (53); 5 to 16
// rows are built as 16 on one CTA of eight warps an SM, which covers too little of the
// latencies: 102 to 125 us.
constexpr int FEW_MOST = 16, FEW_WARPS = 8;
constexpr int few_v(int n) { return n > 4 ? 4 : 8; }   // rows of W of a warp: what the registers allow
constexpr int FEW_X_BYTES = 160 * 1024;   // of the rows of x in shared memory

// GRAD: G of one piece of the vocabulary, as planes, from the same logits: were they
// taken on the tensor cores, which add them up less exactly, the probabilities would
// not add up to one with this lse (gradients of 16 rows of logits of 60 were 2e-5 off).
// With gradient, 50021 x 1024: 4 rows 485 -> 420 us by it, 16 rows 543 -> 542.
struct FewGrad {
    const float4 *grad;       // per kept row, see row_grad
    __nv_bfloat16 *dl;        // [planes][..][pitch]
    int64_t plane;
    int pitch, col0, cols;
};
constexpr int FEW_G_ROWS = BK;   // rows of G that the products read as inner elements

template <int N, int VEC, typename Id, bool GRAD>
__global__ void __launch_bounds__(FEW_WARPS * 32, N > 4 ? 1 : 2)
    k_few_rows(const float *__restrict__ x, const float *__restrict__ W, const void *targets, int n,
               int d, int64_t V, int64_t ignore, float scale2, float2 *part, float *z_target, int2 *row,
               int *kept, const FewGrad grad) {
    extern __shared__ __align__(16) float few_x[];   // [N][pitch], zeros past n and d
    __shared__ int2 rows[FEW_MOST];
    constexpr float NEG_INF = -INFINITY;
    constexpr int FEW_V = few_v(N);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pitch = (d + 32 * VEC - 1) / (32 * VEC) * (32 * VEC);
    dependents_may_launch();
    wait_for_prerequisites();
    int live;
    if (GRAD) {   // numbered by the gathering kernel
        live = *kept;
        if (static_cast<int>(threadIdx.x) < live) rows[threadIdx.x] = row[threadIdx.x];
        // zeros in the rows that the products read besides
        const int pieces = (grad.cols + BK - 1) / BK * (BK / 8);   // of 16 bytes, a row
        for (int i = blockIdx.x * (FEW_WARPS * 32) + threadIdx.x; i < 3 * (FEW_G_ROWS - live) * pieces;
             i += gridDim.x * (FEW_WARPS * 32)) {
            const int r = i / pieces, c = i - r * pieces, pl = r / (FEW_G_ROWS - live);
            const int64_t at = pl * grad.plane + static_cast<int64_t>(live + r - pl * (FEW_G_ROWS - live)) * grad.pitch;
            *reinterpret_cast<uint4 *>(grad.dl + at + c * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncthreads();
    } else {
        live = number_rows<FEW_WARPS * 32, Id>(targets, n, V, ignore, rows);
        if (blockIdx.x == 0) {
            if (static_cast<int>(threadIdx.x) < live) row[threadIdx.x] = rows[threadIdx.x];
            if (threadIdx.x == 0) kept[0] = live, kept[1] = 0;
        }
    }
    for (int i = threadIdx.x; i < N * pitch; i += FEW_WARPS * 32) {
        const int r = i / pitch, c = i - r * pitch;
        few_x[i] = r < live && c < d ? x[static_cast<int64_t>(rows[r].x) * d + c] : 0.f;
    }
    __syncthreads();
    // lane r < N: the reference and sum of row r over this warp's rows of W
    float ref = NEG_INF, sum = 0.f;
    const int my_target = lane < live ? rows[lane].y : -1;
    const float4 mine_grad = GRAD && lane < live ? grad.grad[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t step = static_cast<int64_t>(gridDim.x) * FEW_WARPS * FEW_V;
    const int64_t v_begin = GRAD ? grad.col0 : 0, v_end = GRAD ? v_begin + grad.cols : V;
    const int64_t v_stop = GRAD ? v_begin + (grad.cols + BK - 1) / BK * BK : V;   // zeros from v_end on
    for (int64_t v0 = v_begin + (static_cast<int64_t>(blockIdx.x) * FEW_WARPS + warp) * FEW_V; v0 < v_stop; v0 += step) {
        float G[FEW_V];
        float acc[FEW_V][N];
#pragma unroll
        for (int q = 0; q < FEW_V; ++q)
#pragma unroll
            for (int r = 0; r < N; ++r) acc[q][r] = 0.f;
#pragma unroll 2
        for (int c = lane * VEC; c < pitch; c += 32 * VEC) {
            float w[FEW_V][VEC];
#pragma unroll
            for (int q = 0; q < FEW_V; ++q) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[q][e] = 0.f;
                if (c < d && v0 + q < v_end) load_f32<float, VEC>(W + (v0 + q) * d + c, w[q]);
            }
#pragma unroll
            for (int r = 0; r < N; ++r) {
                float xv[VEC];
                load_f32<float, VEC>(few_x + r * pitch + c, xv);
#pragma unroll
                for (int q = 0; q < FEW_V; ++q)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[q][r] = fmaf(w[q][e], xv[e], acc[q][r]);
            }
        }
        // the lanes' sums: halves are exchanged and added, until lane l has the sums of
        // row r = l / (32 / N) (all its lanes the same)
#pragma unroll
        for (int q = 0; q < FEW_V; ++q) {
            float z[N];
#pragma unroll
            for (int r = 0; r < N; ++r) z[r] = acc[q][r];
#pragma unroll
            for (int o = 16, have = N; o > 0; o >>= 1) {
                if (have > 1) {
                    have /= 2;
                    const bool upper = lane & o;
#pragma unroll
                    for (int r = 0; r < N / 2; ++r) {
                        if (r >= have) break;
                        const float give = upper ? z[r] : z[r + have], keep = upper ? z[r + have] : z[r];
                        z[r] = keep + __shfl_xor_sync(FULL_MASK, give, o);
                    }
                } else {
                    z[0] += __shfl_xor_sync(FULL_MASK, z[0], o);
                }
            }
            // row r's value to lane r
            const float mine = __shfl_sync(FULL_MASK, z[0], (lane % N) * (32 / N));
            if (GRAD) {
                const float p = ex2_approx(fmaf(mine, scale2, -mine_grad.x)) * mine_grad.z;
                G[q] = v0 + q >= v_end ? 0.f : my_target == v0 + q ? p - mine_grad.y : p;
            } else if (lane < N && v0 + q < V) {
                if (my_target == v0 + q) z_target[lane] = mine;
                const float most = fmaxf(ref, mine * scale2);
                const float at = most == NEG_INF ? 0.f : most;
                sum = sum * ex2_approx(ref - at) + ex2_approx(fmaf(mine, scale2, -at));
                ref = most;
            }
        }
        if (GRAD && lane < live) {
            __nv_bfloat16 *to = grad.dl + static_cast<int64_t>(lane) * grad.pitch + (v0 - v_begin);
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) {
                Pack<__nv_bfloat16, FEW_V> o;
#pragma unroll
                for (int q = 0; q < FEW_V; q += 2) {
                    const __nv_bfloat162 h =
                        pl == 0 ? finite_bf16x2(G[q], G[q + 1]) : __floats2bfloat162_rn(G[q], G[q + 1]);
                    o.v[q] = __low2bfloat16(h);
                    o.v[q + 1] = __high2bfloat16(h);
                    G[q] -= __low2float(h);
                    G[q + 1] -= __high2float(h);
                }
                *reinterpret_cast<Pack<__nv_bfloat16, FEW_V> *>(to + pl * grad.plane) = o;
            }
        }
    }
    if (GRAD) return;
    if (lane < live) part[static_cast<int64_t>(lane) * (gridDim.x * FEW_WARPS) + blockIdx.x * FEW_WARPS + warp] = make_float2(ref, sum);
}

// Joins the row's partial maxima and sums; a warp per row.  Rows that take no
// part: zeros (a target out of range: NaN).
template <typename Id>
__global__ void __launch_bounds__(256)
    k_loss_join(const float2 *__restrict__ part, int groups, const float *__restrict__ z_target,
                const int2 *__restrict__ row, const int *__restrict__ kept, const void *targets, int n,
                int64_t V, int64_t ignore, float scale2, float *__restrict__ loss, float *__restrict__ lse) {
    wait_for_prerequisites();
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
        if (lane == 0) {   // one rounding of lse at its own size: the backward's p takes it all
            const float ln_s = logf(s);
            const int i = row[m].x;
            lse[i] = fmaf(mx, LN2, ln_s);
            loss[i] = fmaf(fmaf(-z_target[m], scale2, mx), LN2, ln_s);
        }
    }
    const int64_t id = static_cast<int64_t>(static_cast<const Id *>(targets)[m]);
    if (lane == 0 && (id == ignore || id < 0 || id >= V)) {
        const float v = id == ignore ? 0.f : __int_as_float(0x7fffffff);
        lse[m] = v;
        loss[m] = v;
    }
}

// ---------------------------------------------------------------- host side
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// rows of x that a tile's first CTA reads: below HALF_M rows all there are, since x's
// whole tile would be as much to read as W's (64 rows over 50021 x 1024 bf16, forward:
// 35.7 -> 33.6 us)
int rows_of_x(int64_t n) { return n < HALF_M ? static_cast<int>(ceil_div(n, 8) * 8) : HALF_M; }

// The sizes a call works with, the same for the workspace query and the call.
struct Plan {
    int planes, g_planes, pitch, d_bn, fwd_bn;
    int64_t rows_pad;
    bool copy_w;
    int64_t piece;        // backward: vocabulary rows of a piece
    int pieces, group, groups;
    size_t kept, row, x, w, part, z, grad, dl, parts, acc, total;
};

constexpr int FEW_CTAS = 4 * PAIRS;
int few_size(int64_t n) { return n <= 1 ? 1 : n <= 4 ? 4 : FEW_MOST; }   // rows it is built for

// Bytes the piece of G may take.  More would be faster where it binds, as gx's sums
// pass through memory less often, but the caller pays for it: 262144 rows over 65536 x
// 1024 bf16 with gradient take 122 ms with 1 GiB (32 pieces of 2048), 107 with 2, 97
// with 4.  At least 2048 columns, 32 slices of gx's products.
constexpr int64_t PIECE_BYTES = 1ll << 30;

// Rows up to which a bf16 G is kept as two planes, to 2^-16: the roundings of so few
// rows' largest entries need not average out (4 rows: gx off by up to 1.54 times what
// rounding it costs, 1.00 with two planes).  That is another product of the same
// slices: 64 rows over 50021 x 512 with gradient 87 -> 99 us, 4 over 50021 x 1024 123 ->
// 141.  200 rows over 50021 x 1024 would go from 160 to 188 for 1.2 -> 1.00.
constexpr int TWO_PLANES_MOST = 64;

// Columns of the forward's tiles.  With enough tiles the widest; with few, the width
// that leaves the busiest pair the least to do: a tile costs its columns and, for
// the rows of x that it reads again, about 64 more (4 rows over 50021 x 1024: three
// tiles of 224 a pair instead of three of 256).
int forward_columns(int64_t tiles_m, int64_t V) {
    if (tiles_m * ceil_div(V, BN) >= 8 * PAIRS) return BN;
    int best = BN;
    int64_t least = INT64_MAX;
    for (int bn = BN; bn >= 64; bn -= 32) {
        const int64_t load = ceil_div(tiles_m * ceil_div(V, bn), PAIRS) * (bn + 64);
        if (load < least) {
            least = load;
            best = bn;
        }
    }
    return best;
}

Plan plan_for(int64_t n, int64_t d, int64_t V, int dtype, bool w_aligned, bool backward) {
    Plan p{};
    const bool split = dtype == NRNN_F32;
    p.planes = split ? 3 : 1;
    p.g_planes = split ? 3 : n <= TWO_PLANES_MOST ? 2 : 1;
    p.pitch = static_cast<int>((d + 7) / 8 * 8);
    p.rows_pad = ceil_div(n, BM) * BM;
    p.copy_w = split || d % 8 != 0 || !w_aligned;
    // columns of gx and gW in equal tiles
    p.d_bn = static_cast<int>(ceil_div(ceil_div(d, ceil_div(d, BN)), 32) * 32);
    const int64_t tiles_m = ceil_div(n, BM);
    p.fwd_bn = forward_columns(tiles_m, V);
    const int64_t tiles_v = ceil_div(V, p.fwd_bn);
    // about eight units per pair
    p.group = static_cast<int>(tiles_m * tiles_v / (PAIRS * 8));
    p.group = p.group < 1 ? 1 : p.group > 16 ? 16 : p.group;
    p.groups = static_cast<int>(ceil_div(tiles_v, p.group));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    p.kept = take(3 * sizeof(int));   // {number, error, back}; first of all: the header names the error's place
    p.row = take(sizeof(int2) * n);
    p.x = take(sizeof(__nv_bfloat16) * p.planes * p.rows_pad * p.pitch);
    p.w = take(p.copy_w ? sizeof(__nv_bfloat16) * p.planes * V * p.pitch : 0);
    if (!backward) {
        const int64_t parts = 2 * p.groups > FEW_CTAS * FEW_WARPS || n > FEW_MOST ? 2 * p.groups : FEW_CTAS * FEW_WARPS;
        p.part = take(sizeof(float2) * n * parts);
        p.z = take(sizeof(float) * n);
    } else {
        p.grad = take(sizeof(float4) * n);
        const int64_t all = ceil_div(V, BN) * BN;
        p.piece = PIECE_BYTES / (2 * p.g_planes * p.rows_pad) / BN * BN;
        p.piece = p.piece < 2048 ? 2048 : p.piece;
        p.piece = p.piece > all ? all : p.piece;
        p.pieces = static_cast<int>(ceil_div(V, p.piece));
        p.dl = take(sizeof(__nv_bfloat16) * p.g_planes * p.rows_pad * p.piece);
        p.parts = take(sizeof(float) * 2 * PAIRS * BM * p.d_bn);
        p.acc = take(p.pieces > 1 ? sizeof(float) * p.rows_pad * p.pitch : 0);
    }
    p.total = at;
    return p;
}

template <int FORM, typename T>
cudaError_t gemm(const CUtensorMap &tmA, const CUtensorMap &tmB, const CUtensorMap &tmOut,
                 const GemmArgs &a, int64_t most_units, int64_t tiles, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = once_per_device(configured, [](int) {
        return cudaFuncSetAttribute(k_vocab_gemm<FORM, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(GEMM_SMEM));
    });
    if (e != cudaSuccess) return e;
    if (most_units > INT32_MAX) return cudaErrorInvalidConfiguration;
    const unsigned pairs = static_cast<unsigned>(most_units < PAIRS ? most_units : PAIRS);
    e = launch_dependent(k_vocab_gemm<FORM, T>, 2 * pairs, GEMM_THREADS, GEMM_SMEM, s, tmA, tmB, tmOut, a);
    if constexpr (FORM == GX || FORM == GW) {
        if (e == cudaSuccess && pairs > 1 && most_units > tiles) {   // tiles of several slices
            // tiles that may be cut: those left over by whole waves of any number of kept rows
            const int64_t cut = tiles < pairs ? tiles : pairs;
            const bool few = cut * 8 <= pairs;   // eight parts each and more
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(cut), few ? BM : BM / JOIN_WARPS);
            cfg.blockDim = dim3(JOIN_WARPS * 32);
            cfg.stream = s;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaLaunchKernelEx(&cfg, few ? k_join_parts<FORM, T, true> : k_join_parts<FORM, T, false>, a,
                                   static_cast<int>(pairs));
        }
    }
    return e;
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
    GatherArgs g{};
    g.x = c.x; g.row = row; g.kept = kept;
    g.out = reinterpret_cast<__nv_bfloat16 *>(c.ws + p.x);
    g.rows_pad = p.rows_pad; g.d = static_cast<int>(c.d); g.pitch = p.pitch;
    g.lse = lse; g.gl = gl; g.scale = c.scale;
    g.grad = lse != nullptr ? reinterpret_cast<float4 *>(c.ws + p.grad) : nullptr;
    g.back = reinterpret_cast<float *>(kept + 2);
    g.gx = gx; g.targets = c.targets; g.V = c.V; g.ignore = c.ignore; g.n = static_cast<int>(c.n);
    const int64_t want = p.rows_pad / (GATHER_THREADS / 32);
    const unsigned blocks = static_cast<unsigned>(want < 4864 ? want : 4864);
    cudaError_t e;
    if (c.n <= FEW_ROWS) {
        e = launch_dependent(k_gather_rows<T, Id, true>, blocks, GATHER_THREADS, 0, c.stream, g);
    } else {
        e = launch_dependent(k_kept_rows<Id>, 1, KEPT_THREADS, 0, c.stream, c.targets, static_cast<int>(c.n), c.V,
                             c.ignore, row, kept);
        if (e == cudaSuccess)
            e = launch_dependent(k_gather_rows<T, Id, false>, blocks, GATHER_THREADS, 0, c.stream, g);
    }
    *w_out = c.W;
    if (e == cudaSuccess && p.copy_w) {
        __nv_bfloat16 *w = reinterpret_cast<__nv_bfloat16 *>(c.ws + p.w);
        const int64_t b = ceil_div(c.V, 8);
        e = launch_dependent(k_planes<T>, static_cast<unsigned>(b < 4864 ? b : 4864), 256, 0, c.stream,
                             static_cast<const T *>(c.W), w, c.V, static_cast<int>(c.d), p.pitch);
        *w_out = w;
    }
    return e;
}

// loss and lse from `parts` partial sums a row
template <typename Id> int join_loss(const Call &c, const Plan &p, int parts, float *loss, float *lse) {
    return launch_dependent(k_loss_join<Id>, static_cast<unsigned>(ceil_div(c.n, 8)), 256, 0, c.stream,
                            reinterpret_cast<const float2 *>(c.ws + p.part), parts,
                            reinterpret_cast<const float *>(c.ws + p.z),
                            reinterpret_cast<const int2 *>(c.ws + p.row),
                            reinterpret_cast<const int *>(c.ws + p.kept), c.targets,
                            static_cast<int>(c.n), c.V, c.ignore, c.scale * LOG2E, loss, lse) == cudaSuccess
               ? NRNN_OK : NRNN_ERR_CUDA;
}

// fp32 rows that the few-rows form takes: few, and fit in shared memory
bool few_rows(int64_t n, int64_t d, int dtype) {
    return dtype == NRNN_F32 && n <= FEW_MOST && few_size(n) * (d + 127) * 4 <= FEW_X_BYTES;
}

template <int N, int VEC, typename Id, bool GRAD>
cudaError_t launch_few(const Call &c, const Plan &p, const FewGrad &grad) {
    constexpr int most = FEW_X_BYTES;
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = once_per_device(configured, [](int) {
        return cudaFuncSetAttribute(k_few_rows<N, VEC, Id, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    });
    if (e != cudaSuccess) return e;
    const size_t smem = sizeof(float) * N * (ceil_div(c.d, 32 * VEC) * 32 * VEC);
    return launch_dependent(k_few_rows<N, VEC, Id, GRAD>, FEW_CTAS, FEW_WARPS * 32, smem, c.stream,
                            static_cast<const float *>(c.x), static_cast<const float *>(c.W), c.targets,
                            static_cast<int>(c.n), static_cast<int>(c.d), c.V, c.ignore, c.scale * LOG2E,
                            reinterpret_cast<float2 *>(c.ws + p.part), reinterpret_cast<float *>(c.ws + p.z),
                            reinterpret_cast<int2 *>(c.ws + p.row), reinterpret_cast<int *>(c.ws + p.kept), grad);
}

template <typename Id, bool GRAD> cudaError_t launch_few(const Call &c, const Plan &p, const FewGrad &grad = {}) {
    const bool wide = c.d % 4 == 0 && (reinterpret_cast<uintptr_t>(c.W) & 15) == 0;
    switch (few_size(c.n)) {
        case 1: return wide ? launch_few<1, 4, Id, GRAD>(c, p, grad) : launch_few<1, 1, Id, GRAD>(c, p, grad);
        case 4: return wide ? launch_few<4, 4, Id, GRAD>(c, p, grad) : launch_few<4, 1, Id, GRAD>(c, p, grad);
        default: return wide ? launch_few<16, 4, Id, GRAD>(c, p, grad) : launch_few<16, 1, Id, GRAD>(c, p, grad);
    }
}

template <typename T, typename Id>
int forward(const Call &c, float *loss, float *lse) {
    const Plan p = plan_for(c.n, c.d, c.V, c.dtype, reinterpret_cast<uintptr_t>(c.W) % 16 == 0, false);
    if constexpr (sizeof(T) == 4) {
        if (few_rows(c.n, c.d, c.dtype)) {
            if (launch_few<Id, false>(c, p) != cudaSuccess) return NRNN_ERR_CUDA;
            return join_loss<Id>(c, p, FEW_CTAS * FEW_WARPS, loss, lse);
        }
    }
    const void *w;
    if (lay_out<T, Id>(c, p, nullptr, nullptr, nullptr, &w) != cudaSuccess) return NRNN_ERR_CUDA;
    CUtensorMap tmA, tmB;
    if (!make_map_planes(&tmA, c.ws + p.x, p.pitch, p.rows_pad, p.planes, BK, rows_of_x(c.n), true) ||
        !make_map_planes(&tmB, w, p.pitch, c.V, p.planes, BK, p.fwd_bn / 2, true))
        return NRNN_ERR_CUDA;
    GemmArgs a{};
    a.kept = reinterpret_cast<int *>(c.ws + p.kept);
    a.error = reinterpret_cast<uint32_t *>(c.ws + p.kept) + 1;
    a.wait_ns = wait_limit_ns();
    a.M = -1; a.K = static_cast<int>(c.d);
    a.bn = p.fwd_bn; a.n_cols = static_cast<int>(c.V);
    a.group = p.group;
    a.a_rows = rows_of_x(c.n);
    a.scale = c.scale;
    a.row = reinterpret_cast<int2 *>(c.ws + p.row);
    a.part = reinterpret_cast<float2 *>(c.ws + p.part);
    a.z_target = reinterpret_cast<float *>(c.ws + p.z);
    if (gemm<LSE, T>(tmA, tmB, tmA, a, ceil_div(c.n, BM) * p.groups, 0, c.stream) != cudaSuccess)
        return NRNN_ERR_CUDA;
    return join_loss<Id>(c, p, 2 * p.groups, loss, lse);
}

template <typename T, typename Id>
int backward(const Call &c, const float *lse, const float *gl, void *gx, void *gW) {
    const Plan p = plan_for(c.n, c.d, c.V, c.dtype, reinterpret_cast<uintptr_t>(c.W) % 16 == 0, true);
    const void *w;
    if (lay_out<T, Id>(c, p, lse, gl, gx, &w) != cudaSuccess) return NRNN_ERR_CUDA;
    unsigned char *x = c.ws + p.x, *dl = c.ws + p.dl;
    CUtensorMap xk, wk, gk, wn, gn, xn, gs, ws;   // K-major x, W, G; MN-major W, G, x; stores of G and gW
    constexpr int tile_v = BN;
    if (!make_map_planes(&xk, x, p.pitch, p.rows_pad, p.planes, BK, rows_of_x(c.n), true) ||
        !make_map_planes(&wk, w, p.pitch, c.V, p.planes, BK, tile_v / 2, true) ||
        !make_map_planes(&gk, dl, p.piece, p.rows_pad, p.g_planes, BK, HALF_M, true) ||
        !make_map_planes(&wn, w, p.pitch, c.V, p.planes, 64, BK, true) ||
        !make_map_planes(&gn, dl, p.piece, p.rows_pad, p.g_planes, 64, BK, true) ||
        !make_map_planes(&xn, x, p.pitch, p.rows_pad, p.planes, 64, BK, true) ||
        !make_map_planes(&gs, dl, p.piece, p.rows_pad, p.g_planes, PIECE, BOX_ROWS, true))
        return NRNN_ERR_CUDA;
    // blocks of 64 columns: the tiles have to be whole blocks, so that none reaches into
    // the next tile's columns (past gW's ends TMA writes nothing)
    const bool blocks_out = sizeof(T) == 2 && c.d % 8 == 0 && p.d_bn % PIECE == 0 &&
                            (reinterpret_cast<uintptr_t>(gW) & 15) == 0;
    ws = gs;
    if (blocks_out && !make_map_planes(&ws, gW, c.d, c.V, 1, PIECE, BOX_ROWS, true)) return NRNN_ERR_CUDA;
    GemmArgs a{};
    a.blocks_out = blocks_out;
    a.kept = reinterpret_cast<int *>(c.ws + p.kept);
    a.error = reinterpret_cast<uint32_t *>(c.ws + p.kept) + 1;
    a.wait_ns = wait_limit_ns();
    a.scale = c.scale;
    a.a_rows = rows_of_x(c.n);
    a.row = reinterpret_cast<int2 *>(c.ws + p.row);
    a.grad = reinterpret_cast<float4 *>(c.ws + p.grad);
    a.back = reinterpret_cast<float *>(c.ws + p.kept) + 2;
    a.g_planes = p.g_planes;
    a.d = static_cast<int>(c.d);
    a.parts = reinterpret_cast<float *>(c.ws + p.parts);
    a.acc = reinterpret_cast<float *>(c.ws + p.acc);
    a.acc_pitch = p.pitch;
    const int64_t tiles_m = ceil_div(c.n, BM), tiles_d = ceil_div(c.d, p.d_bn);
    for (int i = 0; i < p.pieces; ++i) {
        const int64_t v0 = i * p.piece;
        const int cols = static_cast<int>(c.V - v0 < p.piece ? c.V - v0 : p.piece);
        a.col0 = static_cast<int>(v0);
        a.M = -1; a.K = static_cast<int>(c.d);
        a.bn = tile_v; a.n_cols = cols;
        cudaError_t e;
        if (few_rows(c.n, c.d, c.dtype)) {   // the form that the forward takes its logits in
            const FewGrad few{a.grad, reinterpret_cast<__nv_bfloat16 *>(dl), p.rows_pad * p.piece,
                              static_cast<int>(p.piece), a.col0, cols};
            e = launch_few<int32_t, true>(c, p, few);   // (reads no ids)
        } else {
            e = gemm<DL, T>(xk, wk, gs, a, tiles_m * ceil_div(cols, tile_v), 0, c.stream);
        }
        if (e != cudaSuccess) return NRNN_ERR_CUDA;
        a.bn = p.d_bn; a.n_cols = a.d;
        a.K = cols;
        a.out = gx;
        a.acc_in = i > 0;
        a.acc_out = i + 1 < p.pieces;
        if (gemm<GX, T>(gk, wn, gs, a, tiles_m * tiles_d * ceil_div(cols, BK),
                        tiles_m * tiles_d, c.stream) != cudaSuccess)
            return NRNN_ERR_CUDA;
        a.M = cols; a.K = -1;
        a.out = gW;
        if (gemm<GW, T>(gn, xn, ws, a, ceil_div(cols, BM) * tiles_d * ceil_div(c.n, BK),
                        ceil_div(cols, BM) * tiles_d, c.stream) != cudaSuccess)
            return NRNN_ERR_CUDA;
    }
    return NRNN_OK;
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
    if (loss == nullptr || lse == nullptr ||
        (reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(lse)) % sizeof(float) != 0)
        return NRNN_ERR_INVALID_ARG;
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
    if ((reinterpret_cast<uintptr_t>(gx) | reinterpret_cast<uintptr_t>(gW)) % elem != 0 ||
        (reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(g_loss)) % sizeof(float) != 0)
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
