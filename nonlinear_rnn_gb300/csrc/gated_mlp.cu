// Gated feed-forward block and its gradient.
//
//   a = x Wg^T, b = x Wu^T, m = silu(a) b, y = m Wo^T        W_in = [Wg; Wu]
//   p = dm/da = b silu'(a), q = dm/db = silu(a)
//   gm = g Wo, ga = gm p, gb = gm q
//   gx = [ga gb] W_in, gW_in = [ga gb]^T x, gW_out = g^T m
//
// 6 n d f operations forward and 12 n d f backward: bound by the tensor cores, except
// for few rows, where reading the weights bounds it.
//
// All products run on one persistent tcgen05 kernel (k_mlp_gemm) of CTA pairs
// (cta_group::2), as the vocabulary loss's: 256 x (up to 256) tiles, TMA into a ring of
// 128-byte-swizzled stages, one thread issuing the products into one of two TMEM
// accumulators while eight epilogue warps drain the other.  Transposed operands are read
// MN-major from where they lie.  The forms:
//   UP   x W_in^T    A pair's two CTAs stage one half each of a tile's columns: one the
//                    rows of Wg, the other the same rows of Wu.  The accumulator then
//                    holds a and b of the same 128 units beside one another, and the
//                    epilogue forms m without either having been stored.  With the
//                    gradient to come p and q are kept: fp32, or for bf16 24 bits of them.
//   DOWN m W_out^T
//   DH   g W_out     gm, from which the epilogue forms ga and gb by the kept p and q
//   GX   [ga gb] W_in          the inner dimension runs over ga, then gb
//   GWI  [ga gb]^T x           rows of gW_in, Wg's tiles, then Wu's
//   GWO  g^T m
//
// UP and DH have many tiles; the others may have few and long inner dimensions.  Where
// these are less than WAVES_UNCUT waves, whole waves of tiles go one to a pair and the
// rest is cut by inner slices, an equal run of the (tile, slice) sequence to every team of
// pairs; parts of a cut tile go to the workspace in fp32 and k_join_parts adds them in
// order.
//
// For bf16, m (formed from unrounded a and b) is rounded before the second product, and
// ga and gb (formed from unrounded gm) before theirs: an operand of the tensor cores is
// bf16, and a second plane of each would double these products.  So every result is 1.41
// times as far off as rounding the exact one once: two roundings.  p and q are no operands
// and keep 16 bits of significand, 2^-15 at most off, as one of 2^-9 more would make gx and
// gW_in 1.73 times as far off.  Up to TWO_PLANES_MOST rows m, ga and gb are two planes all the
// same.
//
// fp32 operands are split into three bf16 planes, v = hi + mid + lo up to 2^-24, and a
// product is the six plane products above 2^-24 relative, smallest first.  An
// accumulator takes at most 256 elements of the inner dimension before the epilogue adds
// it to fp32 registers, as the tensor cores add less exactly than fp32 rounding does.
// (An infinity leaves no number: in fp32 operands it counts as NaN.)
//
// Measured: a training step of 32768 rows of 1024 x 4096 bf16 1.75 to 1.83 ms (1.35 to 1.42 PFLOP/s; the
// kernels apart, of 8192 rows under a profiler: UP 107 us, DOWN 49, DH 70, GX 85, GWI 84, GWO 49).  The forward
// that keeps nothing runs at 1.7 PFLOP/s, the rate of cuBLAS kept up, that is, at the power
// limit; keeping p and q costs 80 us for 0.81 GB.  1501 x 250 x 683 fp32, training: 127 us.
//
// Every wait is bounded.  One that gives up sets the call's error word (the workspace's
// first) and the abort flag of both CTAs of the pair, which ends the other roles' waits
// too; the epilogues write NaN from there on, and neither CTA leaves before what both
// have in flight is done (settle).
#include <type_traits>

#include "../../include/nrnn.h"
#include "nrnn_internal.h"
#include "pair.cuh"

namespace nrnn {
namespace {

constexpr int PAIRS = 76;   // of 152 SMs
constexpr int MOST_SIDE = 8;
constexpr int WAVES_UNCUT = 4;   // a last wave of this many loses less than joining its parts costs

enum Form { UP, DOWN, DH, GX, GWI, GWO };

constexpr int BM = 256, BN = 256, BK = 64;                 // of a pair
constexpr int HALF_M = BM / 2;                             // rows of A and D in one CTA
constexpr int A_BYTES = HALF_M * BK * 2, B_BYTES = BN / 2 * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int GEMM_THREADS = 128 + EPI_WARPS * 32;
constexpr int PIECE = 64;                                  // columns that an epilogue warp takes at a time
constexpr int BOX_ROWS = 32, BOX_BYTES = BOX_ROWS * PIECE * 2;
constexpr int SPLIT_CHUNK = 4;     // fp32: 64-wide slices per accumulator
constexpr int SEGMENTS = 6;        // fp32: plane products, smallest first
__device__ constexpr int PLANE_A[SEGMENTS] = {2, 1, 0, 1, 0, 0};
__device__ constexpr int PLANE_B[SEGMENTS] = {0, 1, 2, 0, 1, 0};

// staged blocks of an epilogue warp, and the stages that they leave room for
template <int FORM, typename T> constexpr int blocks_of() { return sizeof(T) == 2 && FORM == DH ? 2 : 1; }
template <int FORM, typename T> constexpr int stages_of() { return blocks_of<FORM, T>() == 2 ? 5 : 6; }
template <int FORM, typename T> constexpr size_t gemm_smem() {
    return stages_of<FORM, T>() * STAGE_BYTES + EPI_WARPS * blocks_of<FORM, T>() * BOX_BYTES + 1024;
}

struct GemmArgs {
    uint32_t *error;          // device: set by a wait that gave up
    uint64_t wait_ns;         // limit of a wait
    int M, N;                 // rows (GWI: of one half) and columns of the product
    int tiles_m, tiles_n;     // row tiles (GWI: of both halves) and column tiles
    int kb, kb_half;          // 64-wide inner slices; GX: of one half
    int m_half;               // GWI: row tiles of a half
    int bn;                   // columns of a tile: a multiple of 64, at most BN (UP: of both halves)
    int whole, units;         // DOWN, GX, GWI, GWO: row tiles of a team that are not cut, and all
    int side, teams;          // pairs of a team (its column tiles beside one another), teams
    int share, longer;        // slices of cut tiles of a team: share, and one more of the first `longer`
    float *parts;             // [pairs][2][BM][bn] sums of cut tiles
    void *out;                // the result in the storage type, rows of N
    bool blocks_out;          // bf16: tmOut is over the result, whose blocks leave by TMA
    int inner;                // bf16: planes that UP and DH store and the other products take: 1 or 2
    void *pq;                 // p and q: fp32 [2][M][pitch]; bf16 blocks of KEPT_ROWS x KEPT_COLS
    int pitch;
    int kept_cols;            // bf16: blocks beside one another
};

// A unit is what a pair takes at a time: a tile, or a tile's slices k0 .. k1
struct Unit { int tm, tn, k0, k1, slot; };   // slot: -1 = a whole tile

template <int FORM> constexpr bool CUTS = FORM != UP && FORM != DH;

// UP, DH: row tiles that the pairs work on at a time.  Their outputs (p, q and m; ga and
// gb) pass through L2 and push out what lies there, so a band's rows of x are taken while
// they are there (all row tiles against one column tile after another: DH of 32768 x 1024
// x 4096 bf16 280 us, in bands of 8 231; of 4 and 16 the step takes 1% longer).
constexpr int BAND = 8;

template <int FORM> struct Walk {
    int u, pairs, side_at, pos, end;

    __device__ Walk(const GemmArgs &a, int pair, int pairs_) : u(pair), pairs(pairs_), side_at(0), pos(0), end(0) {
        if (!CUTS<FORM>) return;
        side_at = pair % a.side;
        u = pair / a.side;
        if (u < a.teams) run(a, u, pos, end);
        else u = a.units;   // a pair left over
    }
    // the run of team b among the slices of the tiles that are cut
    __device__ static void run(const GemmArgs &a, int b, int &from, int &to) {
        from = b * a.share + min(b, a.longer);
        to = from + a.share + (b < a.longer ? 1 : 0);
    }
    // the team whose run holds a slice
    __device__ static int team_of(const GemmArgs &a, int slice) {
        const int head = a.longer * (a.share + 1);
        return slice < head ? slice / (a.share + 1) : a.longer + (slice - head) / a.share;
    }
    __device__ __forceinline__ bool next(const GemmArgs &a, Unit &t) {
        t.k0 = 0; t.k1 = a.kb; t.slot = -1;
        if (!CUTS<FORM>) {
            if (u >= a.units) return false;
            // bands of row tiles, each against all column tiles, rows fastest
            const int band = u / (BAND * a.tiles_n), in_band = u - band * (BAND * a.tiles_n);
            const int rows = min(BAND, a.tiles_m - band * BAND);
            t.tn = in_band / rows;
            t.tm = band * BAND + in_band - t.tn * rows;
            u += pairs;
            return true;
        }
        int tile = u;
        if (u < a.whole) {
            u += a.teams;
        } else {
            if (pos >= end) return false;
            tile = a.whole + pos / a.kb;
            t.k0 = pos % a.kb;
            if (end - pos < a.kb - t.k0) t.k1 = t.k0 + (end - pos);
            pos += t.k1 - t.k0;
            if (t.k0 > 0) t.slot = 0;
            else if (t.k1 < a.kb) t.slot = 1;
        }
        t.tn = a.side > 1 ? side_at : tile % a.tiles_n;
        t.tm = a.side > 1 ? tile : tile / a.tiles_n;
        return true;
    }
};

__device__ __forceinline__ float sigmoid_of(float x) { return rcp_approx(1.f + ex2_approx(-LOG2E * x)); }

// m = silu(a) b; in place of a and b what the gradient takes: dm/da = b silu'(a) and
// dm/db = silu(a), silu'(a) = s + silu(a) (1 - s)
__device__ __forceinline__ float gate(float &a, float &b) {
    const float s = sigmoid_of(a), q = a * s, m = q * b;
    a = b * fmaf(q, 1.f - s, s);
    b = q;
    return m;
}

// bf16: p and q as kept, without the low 8 of their 32 bits.  A block is 32 rows of 16
// columns, a lane's row in six pieces of 16 bytes, a piece of all lanes side by side: the
// upper halves of p and of q, two pieces each, then the third bytes of p and of q.  So the
// epilogue that forms them and the one that takes them both move whole lines, from and to
// the registers, past what L2 has better use for.  (Rows beyond M and columns beyond N of the
// last blocks hold zeros.)  Against bf16 rows through shared memory, both directions of 8192
// and of 32768 rows over 1024 x 4096: 452 and 1704 us before, 446 and 1694 now, with half as
// many bytes more.
constexpr int KEPT_ROWS = 32, KEPT_COLS = 16, KEPT_PIECES = 6, KEPT_BYTES = KEPT_PIECES * KEPT_ROWS * 16;

// a lane's piece 0 of the block at row y, column x; piece j is KEPT_ROWS j further on
__device__ __forceinline__ uint4 *kept_at(const GemmArgs &a, int y, int x, int lane) {
    return static_cast<uint4 *>(a.pq) +
           (static_cast<int64_t>(y / KEPT_ROWS) * a.kept_cols + x / KEPT_COLS) * (KEPT_BYTES / 16) + lane;
}
__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
// upper halves of 8 values; third bytes of 16
__device__ __forceinline__ uint4 upper_halves(const float *v) {
    return make_uint4(__byte_perm(bits(v[0]), bits(v[1]), 0x7632), __byte_perm(bits(v[2]), bits(v[3]), 0x7632),
                      __byte_perm(bits(v[4]), bits(v[5]), 0x7632), __byte_perm(bits(v[6]), bits(v[7]), 0x7632));
}
__device__ __forceinline__ uint32_t third_bytes_of_4(const float *v) {
    return __byte_perm(__byte_perm(bits(v[0]), bits(v[1]), 0x0051), __byte_perm(bits(v[2]), bits(v[3]), 0x0051), 0x5410);
}
__device__ __forceinline__ uint4 third_bytes(const float *v) {
    return make_uint4(third_bytes_of_4(v), third_bytes_of_4(v + 4), third_bytes_of_4(v + 8), third_bytes_of_4(v + 12));
}
// Two values of a word of upper halves and the bytes k, k + 1 of a word of third bytes.  The
// third byte stands in for the fourth too: zeros, infinities and NaN stay what they are, and
// the dropped bits are replaced by as many on average.
__device__ __forceinline__ float2 kept_pair(uint32_t upper, uint32_t third, int k) {
    return make_float2(__uint_as_float(__byte_perm(upper, third, 0x1000 | (4 + k) * 0x11)),
                       __uint_as_float(__byte_perm(upper, third, 0x3200 | (5 + k) * 0x11)));
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int FORM> __device__ constexpr bool mn_a() { return FORM == GWI || FORM == GWO; }
template <int FORM> __device__ constexpr bool mn_b() { return FORM != UP && FORM != DOWN; }

// bytes of a stage's copies in one CTA: one box of a K-major operand, 64 columns each of
// an MN-major one
template <int FORM> __device__ __forceinline__ uint32_t stage_bytes(const GemmArgs &a) {
    const int half_n = a.bn / 2, b_rows = mn_b<FORM>() ? (half_n + 63) / 64 * 64 : half_n;
    return A_BYTES + b_rows * BK * 2;
}

// T: storage type of the inputs (float: split products).  KEEP: UP stores p and q (apart, as
// what keeps them would cost a forward that does not 3%)
template <int FORM, typename T, bool KEEP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GEMM_THREADS, 1)
    k_mlp_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmOut, const GemmArgs a) {
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr bool MN_A = mn_a<FORM>(), MN_B = mn_b<FORM>();
    constexpr int STAGES = stages_of<FORM, T>(), BLOCKS = blocks_of<FORM, T>();
    constexpr uint32_t TMEM_COLS = 512;   // two accumulators
    extern __shared__ unsigned char dsmem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES], accf_bar[2], acce_bar[2], drain_bar;
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
        prefetch_tensormap(&tmOut);
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
    const int again = !SPLIT && CUTS<FORM> ? a.inner : 1;   // products of a slice, one a plane
    const int half_n = a.bn / 2;
    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        // Lane i starts the i-th copy of a stage.
        constexpr int BOXES_A = MN_A ? HALF_M / 64 : 1;
        const int boxes_b = MN_B ? (half_n + 63) / 64 : 1;
        const uint32_t bytes = 2 * stage_bytes<FORM>(a);
        const bool is_a = lane < BOXES_A, copies = lane < BOXES_A + boxes_b;
        const int box = is_a ? lane : lane - BOXES_A;
        const bool mn = is_a ? MN_A : MN_B;
        const uint32_t offset = (is_a ? 0 : A_BYTES) + box * (64 * BK * 2);
        int it = 0;
        bool go = true;
        while (go && w.next(a, t)) {
            // this lane's coordinate along M or N, and the half of an operand that has two
            int at, half = 0;
            if (is_a) {
                const int tm = FORM == GWI && t.tm >= a.m_half ? t.tm - a.m_half : t.tm;
                half = FORM == GWI && t.tm >= a.m_half;
                at = tm * BM + static_cast<int>(rank) * HALF_M + box * 64;
            } else if (FORM == UP) {
                at = t.tn * half_n;
                half = static_cast<int>(rank);
            } else {
                at = t.tn * a.bn + static_cast<int>(rank) * half_n + box * 64;
            }
            // operands of two halves: plane p of half h is 2 p + h
            constexpr bool TWO_A = FORM == GX || FORM == GWI, TWO_B = FORM == UP || FORM == GX;
            const bool two = is_a ? TWO_A : TWO_B;
            // bf16: whether this lane's operand is one of so many planes, the smaller first
            const bool in_planes = is_a == (FORM != GWO);
            for (int c0 = t.k0; go && c0 < t.k1;) {
                const int c1 = SPLIT && c0 + SPLIT_CHUNK < t.k1 ? c0 + SPLIT_CHUNK : t.k1;
                for (int p = 0; go && p < PASSES; ++p) {
                    int plane = SPLIT ? (is_a ? PLANE_A[p] : PLANE_B[p]) : 0;
                    for (int i = 0; i < (c1 - c0) * again; ++i, ++it) {
                        int k = c0 + i;
                        if (!SPLIT && again == 2) {
                            k = c0 + (i >> 1);
                            plane = in_planes ? 1 - (i & 1) : 0;
                        }
                        const int s = it % STAGES;
                        if (it >= STAGES)
                            go = __all_sync(FULL_MASK, wait_or_abort(a, &empty_bar[s], ((it / STAGES) - 1) & 1, &s_abort));
                        if (!go) break;
                        if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&full_bar[s], bytes);
                        __syncwarp();
                        const bool second = FORM == GX && k >= a.kb_half;
                        const int along_k = (second ? k - a.kb_half : k) * BK;
                        const int z = two ? 2 * plane + (FORM == GX ? (second ? 1 : 0) : half) : plane;
                        if (copies)
                            tma_load_3d_pair(smem + s * STAGE_BYTES + offset, is_a ? &tmA : &tmB,
                                             cluster_addr(&full_bar[s], 0), mn ? at : along_k, mn ? along_k : at, z);
                    }
                }
                c0 = c1;
            }
        }
        if (lane == 0) cluster_store(cluster_addr(const_cast<const int *>(&s_issued[rank]), 0), static_cast<uint32_t>(it));
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc = idesc_bf16(BM, MN_A, MN_B) | static_cast<uint32_t>(a.bn >> 3) << 17;
        int it = 0, phase = 0;
        bool go = true;
        while (go && w.next(a, t)) {
            for (int c0 = t.k0; go && c0 < t.k1; ++phase) {
                const int c1 = SPLIT && c0 + SPLIT_CHUNK < t.k1 ? c0 + SPLIT_CHUNK : t.k1;
                const int buf = phase & 1;
                if (phase >= 2) go = wait_or_abort(a, &acce_bar[buf], ((phase >> 1) - 1) & 1, &s_abort);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + buf * BN;
                const int its = (c1 - c0) * PASSES * again;
                for (int i = 0; go && i < its; ++i, ++it) {
                    const int s = it % STAGES;
                    go = wait_or_abort(a, &full_bar[s], (it / STAGES) & 1, &s_abort);
                    if (!go) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t sa = smem_u32(smem + s * STAGE_BYTES), sb = sa + A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        // 16 elements of K: 32 bytes of a K-major row, or 16 128-byte lines
                        const uint64_t da = MN_A ? sw128_mn_desc(sa + kk * 2048, 64 * BK * 2) : sw128_desc(sa + kk * 32);
                        const uint64_t db = MN_B ? sw128_mn_desc(sb + kk * 2048, 64 * BK * 2) : sw128_desc(sb + kk * 32);
                        mma_f16_pair(d, da, db, idesc, i > 0 || kk > 0 ? 1u : 0u);
                    }
                    mma_commit_pair(&empty_bar[s]);
                }
                if (go) mma_commit_pair(&accf_bar[buf]);
                c0 = c1;
            }
        }
    } else if (warp >= 4) {
        // --------------------------------------------------------------- epilogue
        // warps 4..7 take the even pieces of their 32 rows, 8..11 the odd ones
        const int quarter = warp & 3, odd = (warp - 4) >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        unsigned char *stage_out = smem + STAGES * STAGE_BYTES + (warp - 4) * BLOCKS * BOX_BYTES;
        const float nan = __int_as_float(0x7fffffff);
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
        // block i of this warp: 16-byte piece q of this thread's row, 128-byte swizzle
        auto place = [&](int i, int q) {
            return reinterpret_cast<uint4 *>(stage_out + i * BOX_BYTES + lane * 128 + 16 * (q ^ (lane & 7)));
        };
        auto blocks_free = [&]() {   // the stores before have read the blocks
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
        };
        auto to_bf16 = [](const float *v) {
            uint4 pk;
            uint32_t *o = reinterpret_cast<uint32_t *>(&pk);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                o[e] = *reinterpret_cast<const uint32_t *>(&h);
            }
            return pk;
        };
        auto less_first_plane = [](float *v) {   // 8 values less what to_bf16 makes of them (an infinity: zero)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = __bfloat162float(__float2bfloat16_rn(v[e]));
                v[e] = isinf(h) ? 0.f : v[e] - h;
            }
        };
        // 32 columns of this warp's 32 rows to `to`, rows of `pitch` elements: by way of the
        // block, so that a store takes whole lines (each lane its own row: 4.3 us a CTA for
        // a tile's fp32 parts).  n columns are stored, of `rows` rows; wide: fours at a time
        auto store_32 = [&](const float *v, auto *to, int64_t pitch, int rows, int n, bool wide) {
            using O = std::remove_pointer_t<decltype(to)>;
#pragma unroll
            for (int q = 0; q < 8; ++q) *place(0, q) = *reinterpret_cast<const uint4 *>(v + 4 * q);
            __syncwarp();
            if (wide) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = 4 * k + (lane >> 3), q = lane & 7;
                    if (r < rows && 4 * q < n) {
                        float o[4];
                        load_f32<float, 4>(reinterpret_cast<const float *>(stage_out + r * 128 + 16 * (q ^ (r & 7))), o);
                        store_f32<O, 4>(to + r * pitch + 4 * q, o);
                    }
                }
            } else {
#pragma unroll 8
                for (int r = 0; r < 32; ++r)
                    if (r < rows && lane < n)
                        to[r * pitch + lane] = from_f32<O>(
                            *reinterpret_cast<const float *>(stage_out + r * 128 + 16 * ((lane >> 2) ^ (r & 7)) + 4 * (lane & 3)));
            }
            __syncwarp();
        };
        // the three planes of a piece, v is used up, to column x, row y, planes z, z + dz, z + 2 dz
        auto store_planes = [&](float (&v)[PIECE], int x, int y, int z, int dz) {
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) {
                blocks_free();
#pragma unroll
                for (int q = 0; q < PIECE / 8; ++q) {
                    uint4 pk;
                    uint32_t *o = reinterpret_cast<uint32_t *>(&pk);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &lo = v[q * 8 + 2 * e], &hi = v[q * 8 + 2 * e + 1];
                        const __nv_bfloat162 h2 = pl == 0 ? finite_bf16x2(lo, hi) : __floats2bfloat162_rn(lo, hi);
                        o[e] = *reinterpret_cast<const uint32_t *>(&h2);
                        lo -= __low2float(h2);
                        hi -= __high2float(h2);
                    }
                    *place(0, q) = pk;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && y < a.M) {
                    tma_store_3d(&tmOut, stage_out, x, y, z + pl * dz);
                    bulk_commit();
                }
            }
        };
        while (w.next(a, t)) {
            const int in_tile = static_cast<int>(rank) * HALF_M + quarter * 32;   // the warp's first row
            const bool second = FORM == GWI && t.tm >= a.m_half;
            const int y0 = (second ? t.tm - a.m_half : t.tm) * BM + in_tile;      // in its half
            const int m = y0 + lane;                                              // this thread's row
            auto read32 = [&](int buf, int col, float (&v)[32]) {
                uint32_t r[32];
                tmem_ld_cols<32>(tmem + lane_base + buf * BN + col, r);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = ok ? __uint_as_float(r[e]) : nan;
            };
            // a piece of a plain product's tile
            auto take = [&](int c, float (&v)[PIECE]) {
                const int left = min(a.N - t.tn * a.bn, a.bn) - c, n = min(left, PIECE);
                if (left <= 0) return;
                if (t.slot >= 0) {
                    float *to = a.parts + ((static_cast<int64_t>(pair) * 2 + t.slot) * BM + in_tile) * a.bn + c;
                    blocks_free();
                    store_32(v, to, a.bn, 32, 32, true);
                    store_32(v + 32, to + 32, a.bn, 32, 32, true);
                } else if (!SPLIT && a.blocks_out) {
                    blocks_free();
#pragma unroll
                    for (int q = 0; q < PIECE / 8; ++q) *place(0, q) = to_bf16(v + 8 * q);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && y0 < a.M) {
                        tma_store_3d(&tmOut, stage_out, t.tn * a.bn + c, y0, second ? 1 : 0);
                        bulk_commit();
                    }
                } else if (y0 < a.M) {
                    T *to = static_cast<T *>(a.out) + ((second ? a.M : 0) + static_cast<int64_t>(y0)) * a.N + t.tn * a.bn + c;
                    const bool wide = SPLIT && a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
                    blocks_free();
                    store_32(v, to, a.N, a.M - y0, n, wide);
                    if (n > 32) store_32(v + 32, to + 32, a.N, a.M - y0, n - 32, wide);
                }
            };
            if constexpr (SPLIT) {
                // UP: a piece of a and the same one of b; DH: one piece; else two pieces
                constexpr int PIECES = FORM == DH ? 1 : 2;
                float acc[PIECES][PIECE];
                auto column = [&](int i) { return FORM == UP ? i * half_n + odd * PIECE : (2 * i + odd) * PIECE; };
                const bool mine = FORM != UP || odd * PIECE < half_n;
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
                        for (int h = 0; h < PIECE; h += 32)
                            if (mine && column(i) + h < a.bn) {
                                float v[32];
                                read32(buf, column(i) + h, v);
#pragma unroll
                                for (int e = 0; e < 32; ++e) acc[i][h + e] += v[e];
                            }
                    release(buf);
                }
                if constexpr (FORM == UP) {
                    const int x = t.tn * half_n + odd * PIECE, left = a.N - x;
                    if (mine && left > 0) {
                        if (KEEP && y0 < a.M) {
                            float *p = static_cast<float *>(a.pq) + static_cast<int64_t>(y0) * a.pitch + x,
                                  *q = p + static_cast<int64_t>(a.M) * a.pitch;
                            blocks_free();
#pragma unroll
                            for (int h = 0; h < 2 * PIECE; h += 32) {   // p, then q
                                float v[32];
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    float vp = acc[0][h % PIECE + e], vq = acc[1][h % PIECE + e];
                                    gate(vp, vq);
                                    v[e] = h < PIECE ? vp : vq;
                                }
                                store_32(v, (h < PIECE ? p : q) + h % PIECE, a.pitch, a.M - y0, a.pitch - x - h % PIECE, true);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) acc[0][e] = gate(acc[0][e], acc[1][e]);
                        store_planes(acc[0], x, y0, 0, 1);
                    }
                } else if constexpr (FORM == DH) {
                    const int x = t.tn * a.bn + odd * PIECE, left = a.N - x;
                    if (odd * PIECE < a.bn && left > 0) {
                        float gb[PIECE];
                        const float *pa = static_cast<const float *>(a.pq) + static_cast<int64_t>(m) * a.pitch + x, *pb = pa + static_cast<int64_t>(a.M) * a.pitch;
#pragma unroll
                        for (int q = 0; q < PIECE; q += 4) {
                            float va[4] = {}, vb[4] = {};
                            if (m < a.M && q < left) {   // (the pitch is a multiple of 8: whole fours)
                                load_f32<float, 4>(pa + q, va);
                                load_f32<float, 4>(pb + q, vb);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                gb[q + e] = acc[0][q + e] * vb[e];
                                acc[0][q + e] *= va[e];
                            }
                        }
                        store_planes(acc[0], x, y0, 0, 2);
                        store_planes(gb, x, y0, 1, 2);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < PIECES; ++i)
                        if (column(i) < a.bn) take(column(i), acc[i]);
                }
            } else if (FORM == UP) {
                const int buf = phase & 1, x = t.tn * half_n + odd * PIECE;
                accumulator(buf, (phase >> 1) & 1);
                ++phase;
                if (odd * PIECE >= half_n || x >= a.N) {
                    release(buf);
                    continue;
                }
                // (a second plane of m: the same once more)
#pragma unroll 1
                for (int plane = 0; plane < a.inner; ++plane) {
                    blocks_free();
#pragma unroll
                    for (int h = 0; h < PIECE; h += 32) {
                        float va[32], vb[32];
                        read32(buf, odd * PIECE + h, va);
                        read32(buf, half_n + odd * PIECE + h, vb);
                        if (h + 32 == PIECE && plane + 1 == a.inner) release(buf);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float vm[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) vm[e] = gate(va[8 * q + e], vb[8 * q + e]);
                            if (plane > 0) less_first_plane(vm);
                            *place(0, h / 8 + q) = to_bf16(vm);
                        }
                        if (KEEP && plane == 0 && y0 < a.M) {
#pragma unroll
                            for (int u = 0; u < 32; u += KEPT_COLS)
                                if (x + h + u < a.N) {
                                    uint4 *to = kept_at(a, y0, x + h + u, lane);
                                    __stcs(&to[0], upper_halves(va + u));
                                    __stcs(&to[KEPT_ROWS], upper_halves(va + u + 8));
                                    __stcs(&to[2 * KEPT_ROWS], upper_halves(vb + u));
                                    __stcs(&to[3 * KEPT_ROWS], upper_halves(vb + u + 8));
                                    __stcs(&to[4 * KEPT_ROWS], third_bytes(va + u));
                                    __stcs(&to[5 * KEPT_ROWS], third_bytes(vb + u));
                                }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && y0 < a.M) {
                        tma_store_3d(&tmOut, stage_out, x, y0, plane);
                        bulk_commit();
                    }
                }
            } else if (FORM == DH) {
                const int buf = phase & 1;
                // p and q of two blocks, 32 columns ahead of the products
                uint4 kept[2][KEPT_PIECES] = {};
                auto fetch = [&](int u, int x) {
                    if (x >= a.N || y0 >= a.M) return;
                    const uint4 *from = kept_at(a, y0, x, lane);
#pragma unroll
                    for (int j = 0; j < KEPT_PIECES; ++j) kept[u][j] = __ldcs(from + j * KEPT_ROWS);
                };
                if (odd * PIECE < a.bn)
#pragma unroll
                    for (int u = 0; u < 2; ++u) fetch(u, t.tn * a.bn + odd * PIECE + u * KEPT_COLS);
#pragma unroll 1
                for (int c = odd * PIECE; c < a.bn; c += 2 * PIECE) {
                    const int x = t.tn * a.bn + c;
                    const bool inside = x < a.N && y0 < a.M;
                    if (c < 2 * PIECE) accumulator(buf, (phase >> 1) & 1);
#pragma unroll 1
                    for (int plane = 0; inside && plane < a.inner; ++plane) {
                        const bool last = plane + 1 == a.inner;
                        blocks_free();
#pragma unroll
                        for (int h = 0; h < PIECE; h += 32) {
                            float g[32];
                            read32(buf, c + h, g);
                            if (h + 32 == PIECE && c + 2 * PIECE >= a.bn && last) release(buf);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
#pragma unroll
                                for (int q = 0; q < 2; ++q) {   // 8 columns
                                    const float *gq = g + u * KEPT_COLS + 8 * q;
                                    float va[8], vb[8];
#pragma unroll
                                    for (int e = 0; e < 8; e += 2) {
                                        const float2 p2 = kept_pair(word_of(kept[u][q], e / 2), word_of(kept[u][4], 2 * q + e / 4), e % 4);
                                        const float2 q2 = kept_pair(word_of(kept[u][2 + q], e / 2), word_of(kept[u][5], 2 * q + e / 4), e % 4);
                                        va[e] = p2.x * gq[e];
                                        va[e + 1] = p2.y * gq[e + 1];
                                        vb[e] = q2.x * gq[e];
                                        vb[e + 1] = q2.y * gq[e + 1];
                                    }
                                    if (plane > 0) {
                                        less_first_plane(va);
                                        less_first_plane(vb);
                                    }
                                    *place(0, h / 8 + 2 * u + q) = to_bf16(va);
                                    *place(1, h / 8 + 2 * u + q) = to_bf16(vb);
                                }
                                if (h + 32 < PIECE) fetch(u, x + 32 + u * KEPT_COLS);
                                else if (!last) fetch(u, x + u * KEPT_COLS);
                                else if (c + 2 * PIECE < a.bn) fetch(u, x + 2 * PIECE + u * KEPT_COLS);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_3d(&tmOut, stage_out, x, y0, 2 * plane);
                            tma_store_3d(&tmOut, stage_out + BOX_BYTES, x, y0, 2 * plane + 1);
                            bulk_commit();
                        }
                    }
                    if (!inside && c + 2 * PIECE >= a.bn) release(buf);
                }
                if (odd * PIECE >= a.bn) {
                    accumulator(buf, (phase >> 1) & 1);
                    release(buf);
                }
                ++phase;
            } else {
                const int buf = phase & 1;
                accumulator(buf, (phase >> 1) & 1);
#pragma unroll 1
                for (int c = odd * PIECE; c < a.bn; c += 2 * PIECE) {
                    float v[PIECE];
                    {
                        uint32_t r[PIECE];
                        tmem_ld_cols<PIECE>(tmem + lane_base + buf * BN + c, r);
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) v[e] = ok ? __uint_as_float(r[e]) : nan;
                    }
                    if (c + 2 * PIECE >= a.bn) release(buf);   // the last piece is in registers
                    take(c, v);
                }
                if (odd * PIECE >= a.bn) release(buf);
                ++phase;
            }
        }
        if (lane == 0) bulk_wait_all();   // the stores are done before the CTA exits
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync_all();   // neither CTA leaves while the other may still reach into it
    if (s_abort != 0) {   // the same in both
        if (warp == 1 && lane == 0) {
            if (rank == 0) settle<STAGES>(a, s_issued, full_bar, &drain_bar, stage_bytes<FORM>(a));
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

// Adds the parts of the tiles that a launch of `pairs` pairs cut, in the order of their
// slices.  blockIdx.x: a cut tile; blockIdx.y: JOIN_ROWS of its rows; a thread takes four
// columns of JOIN_EACH rows, its loads JOIN_AHEAD parts ahead.  (Backward of 300 and of 8192
// rows over 1024 x 4096 bf16: 1 row, 8 ahead 72 and 306 us; 2 and 4 67 and 295; 4 and 4 67 and 298.)
constexpr int JOIN_THREADS = 256, JOIN_EACH = 2, JOIN_AHEAD = 4, JOIN_ROWS = JOIN_THREADS / (BN / 4) * JOIN_EACH;

template <int FORM, typename T>
__global__ void __launch_bounds__(JOIN_THREADS) k_join_parts(const GemmArgs a) {
    constexpr int APART = JOIN_THREADS / (BN / 4);   // rows between a thread's
    const int cut = blockIdx.x / a.side, tile = a.whole + cut, side_at = blockIdx.x % a.side;
    const int row = blockIdx.y * JOIN_ROWS + threadIdx.x / (BN / 4), c = threadIdx.x % (BN / 4) * 4;
    const int tm = a.side > 1 ? tile : tile / a.tiles_n, tn = a.side > 1 ? side_at : tile % a.tiles_n;
    const bool second = FORM == GWI && tm >= a.m_half;
    const int m = (second ? tm - a.m_half : tm) * BM + row;
    // the teams whose runs hold slices of this tile: b0 .. b1 (those without a slice are last)
    const int b0 = Walk<FORM>::team_of(a, cut * a.kb), b1 = Walk<FORM>::team_of(a, cut * a.kb + a.kb - 1);
    const int n = min(min(a.bn, a.N - tn * a.bn) - c, 4);
    dependents_may_launch();
    wait_for_prerequisites();
    if (b0 == b1 || m >= a.M || n <= 0) return;   // (one run has it whole)
    const int64_t step = static_cast<int64_t>(2) * BM * a.bn * a.side;   // to the next team's
    const float *p = a.parts + b0 * step + (static_cast<int64_t>(side_at) * 2 * BM + row) * a.bn + c;
    const int apart = APART * a.bn;
    float v[JOIN_EACH][4];
#pragma unroll
    for (int j = 0; j < JOIN_EACH; ++j)   // the first run's part begins with the tile: slot 1
        load_f32<float, 4>(p + static_cast<int64_t>(BM) * a.bn + j * apart, v[j]);
    p += step;
    for (int left = b1 - b0; left > 0; left -= JOIN_AHEAD) {
        float x[JOIN_AHEAD][JOIN_EACH][4];
#pragma unroll
        for (int i = 0; i < JOIN_AHEAD; ++i, p += step)
            if (i < left)
#pragma unroll
                for (int j = 0; j < JOIN_EACH; ++j) load_f32<float, 4>(p + j * apart, x[i][j]);
#pragma unroll
        for (int i = 0; i < JOIN_AHEAD; ++i)
            if (i < left)
#pragma unroll
                for (int j = 0; j < JOIN_EACH; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][e] += x[i][j][e];
    }
    T *to = static_cast<T *>(a.out) + ((second ? a.M : 0) + static_cast<int64_t>(m)) * a.N + tn * a.bn + c;
    const bool wide = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % (4 * sizeof(T)) == 0;
#pragma unroll
    for (int j = 0; j < JOIN_EACH; ++j, to += static_cast<int64_t>(APART) * a.N) {
        if (m + j * APART >= a.M) break;
        if (wide) {
            store_f32<T, 4>(to, v[j]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) to[e] = from_f32<T>(v[j][e]);
        }
    }
}

// The operands that are not used where they lie as (planes, rows, pitch) bf16, zeros
// beyond column d, in one launch; it also clears the call's error word.
struct Copies {
    const void *src[4];
    __nv_bfloat16 *to[4];
    int64_t rows[4];          // 0: none
    int d[4], pitch[4];
    uint32_t *error;
};

template <typename T>
__global__ void __launch_bounds__(256) k_planes(const Copies c) {
    dependents_may_launch();
    wait_for_prerequisites();
    if (blockIdx.x == 0 && threadIdx.x == 0) *c.error = 0;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    int64_t r = blockIdx.x * 8 + (threadIdx.x >> 5);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool wide = wide_rows<T>(c.src[i], c.d[i]);
        for (; r < c.rows[i]; r += warps)
            copy_row<T>(static_cast<const T *>(c.src[i]) + r * c.d[i], c.to[i] + r * c.pitch[i], c.rows[i] * c.pitch[i], c.d[i],
                        c.pitch[i], threadIdx.x & 31, wide);
        r -= c.rows[i];
    }
}

// ---------------------------------------------------------------- few rows
// The rows of a decode step (nothing kept): the weights are read once, and the time is
// their bytes' and latency.  m stays fp32, or two bf16 planes of it (2^-16).
//
// bf16 of aligned rows, up to SHORT_MOST rows of x: the weights' rows are the 16 rows of
// mma.sync products (the 128 rows of tcgen05 would leave most SMs without a tile: 27 us
// for 8 rows over 1024 x 4096).  A lane takes 16 bytes, 8 inner elements, of a row at a
// time, of the weights and of x alike: inner elements may be summed in any order, so
// these are the fragments of two products as they lie.  k_short_up: the 16 rows are 8
// units' rows of Wg and of Wu, so a lane ends with a and b of the same unit and row of x;
// a CTA's warps share the inner dimension.  k_short_down has its first weights under way
// before it waits for m.  8 rows over 1024 x 4096 bf16 (25 MB, 3.7 us of HBM) take 9.3 us
// in a graph, 16 rows 14.
constexpr int SHORT_MOST = 16, SHORT_AHEAD = 4, UP_WARPS = 8, DOWN_WARPS = 16;

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 inner elements of 16 rows (lo: this lane's of rows 0..7, hi: 8..15) and 8 columns
__device__ __forceinline__ void mma_32(float (&c)[4], const uint4 &lo, const uint4 &hi, const uint4 &b) {
    mma_16x8x16(c, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
    mma_16x8x16(c, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// TILES: groups of 8 rows of x
template <int TILES>
__global__ void __launch_bounds__(UP_WARPS * 32)
    k_short_up(const __nv_bfloat16 *__restrict__ x, const __nv_bfloat16 *__restrict__ W, __nv_bfloat16 *__restrict__ m,
               uint32_t *error, int n, int d, int f) {
    __shared__ float share[UP_WARPS][TILES][16][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane >> 2, k0 = lane % 4 * 8, j0 = blockIdx.x * 8;
    wait_for_prerequisites();
    dependents_may_launch();   // (after the wait: the next kernel reads weights before its own)
    if (blockIdx.x == 0 && threadIdx.x == 0) *error = 0;
    const __nv_bfloat16 *gate_row = W + static_cast<int64_t>(min(j0 + row, f - 1)) * d + k0,
                        *up_row = gate_row + static_cast<int64_t>(f) * d;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float c[TILES][4] = {};
    for (int k = warp * 32; k < d; k += UP_WARPS * 32 * SHORT_AHEAD) {
        uint4 lo[SHORT_AHEAD], hi[SHORT_AHEAD], b[SHORT_AHEAD][TILES];
#pragma unroll
        for (int i = 0; i < SHORT_AHEAD; ++i) {
            const int at = k + i * UP_WARPS * 32;
            const bool in = at + k0 < d;   // (d is a multiple of 8)
            lo[i] = in ? *reinterpret_cast<const uint4 *>(gate_row + at) : zero;
            hi[i] = in ? *reinterpret_cast<const uint4 *>(up_row + at) : zero;
#pragma unroll
            for (int t = 0; t < TILES; ++t)
                b[i][t] = in && t * 8 + row < n
                              ? *reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(t * 8 + row) * d + k0 + at) : zero;
        }
#pragma unroll
        for (int i = 0; i < SHORT_AHEAD; ++i)
#pragma unroll
            for (int t = 0; t < TILES; ++t) mma_32(c[t], lo[i], hi[i], b[i][t]);
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
        *reinterpret_cast<float2 *>(&share[warp][t][row][lane % 4 * 2]) = make_float2(c[t][0], c[t][1]);
        *reinterpret_cast<float2 *>(&share[warp][t][row + 8][lane % 4 * 2]) = make_float2(c[t][2], c[t][3]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < TILES * 64; i += UP_WARPS * 32) {
        const int unit = i % 8, col = i / 8 % 8, t = i / 64, r = t * 8 + col;   // r: row of x
        float va = 0.f, vb = 0.f;
#pragma unroll
        for (int w = 0; w < UP_WARPS; ++w) {
            va += share[w][t][unit][col];
            vb += share[w][t][unit + 8][col];
        }
        if (r < n && j0 + unit < f) {
            const float v = gate(va, vb);
            const __nv_bfloat16 h = __float2bfloat16_rn(v);
            const int64_t to = static_cast<int64_t>(r) * f + j0 + unit;
            m[to] = h;
            m[to + static_cast<int64_t>(n) * f] = __float2bfloat16_rn(v - __bfloat162float(h));
        }
    }
}

template <int TILES>
__global__ void __launch_bounds__(DOWN_WARPS * 32)
    k_short_down(const __nv_bfloat16 *__restrict__ m, const __nv_bfloat16 *__restrict__ W, __nv_bfloat16 *__restrict__ y,
                 int n, int d, int f) {
    __shared__ float share[DOWN_WARPS][TILES][16][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane >> 2, k0 = lane % 4 * 8, j0 = blockIdx.x * 16;
    const __nv_bfloat16 *low = W + static_cast<int64_t>(min(j0 + row, d - 1)) * f + k0,
                        *high = W + static_cast<int64_t>(min(j0 + row + 8, d - 1)) * f + k0;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 lo[SHORT_AHEAD], hi[SHORT_AHEAD];
    int k = warp * 32;
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < SHORT_AHEAD; ++i) {
            const int at = k + i * DOWN_WARPS * 32;
            const bool in = at + k0 < f;
            lo[i] = in ? *reinterpret_cast<const uint4 *>(low + at) : zero;
            hi[i] = in ? *reinterpret_cast<const uint4 *>(high + at) : zero;
        }
    };
    fetch();   // the kernel before writes no weights, and those before it are done
    wait_for_prerequisites();
    dependents_may_launch();
    float c[TILES][4] = {};
    const int64_t plane = static_cast<int64_t>(n) * f;
    while (k < f) {
#pragma unroll
        for (int i = 0; i < SHORT_AHEAD; ++i) {
            const int at = k + i * DOWN_WARPS * 32;
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                const bool in = at + k0 < f && t * 8 + row < n;
                const __nv_bfloat16 *from = m + static_cast<int64_t>(t * 8 + row) * f + k0 + at;
                const uint4 b = in ? *reinterpret_cast<const uint4 *>(from) : zero;
                const uint4 b_low = in ? *reinterpret_cast<const uint4 *>(from + plane) : zero;
                mma_32(c[t], lo[i], hi[i], b_low);
                mma_32(c[t], lo[i], hi[i], b);
            }
        }
        k += DOWN_WARPS * 32 * SHORT_AHEAD;
        if (k < f) fetch();
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
        *reinterpret_cast<float2 *>(&share[warp][t][row][lane % 4 * 2]) = make_float2(c[t][0], c[t][1]);
        *reinterpret_cast<float2 *>(&share[warp][t][row + 8][lane % 4 * 2]) = make_float2(c[t][2], c[t][3]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < TILES * 128; i += DOWN_WARPS * 32) {
        const int j = i % 16, col = i / 16 % 8, t = i / 128, r = t * 8 + col;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < DOWN_WARPS; ++w) v += share[w][t][j][col];
        if (r < n && j0 + j < d) y[static_cast<int64_t>(r) * d + j0 + j] = __float2bfloat16_rn(v);
    }
}

// Other types and rows: on the fp32 cores, in groups of FEW_GROUP rows that read the
// weights again, from L2; one group of bf16, FEW_MOST rows of fp32, whose weights'
// planes would be more to write and read (1024 x 4096: 8 rows 12 us, 32 37, 64 69, by the
// planes 111).  A group's rows of x have to fit in FEW_X_BYTES: with 5 rows and more d is at
// most 2817, with 2 to 4 at most 5889; wider ones go by the planes.  A warp of k_few_up takes
// UP_UNITS units at a time, the rows of Wg and Wu of each against every row of x from
// shared memory; a CTA of k_few_down takes DOWN_ROWS rows of W_out, its warps a share of
// the inner dimension each.
constexpr int FEW_GROUP = 8, FEW_MOST = 64, FEW_THREADS = 256, UP_UNITS = 2, FEW_AHEAD = 2;
constexpr size_t FEW_X_BYTES = 96 * 1024;   // of the rows of x in shared memory
constexpr int DOWN_ROWS = 4;

// Sums over the lanes of V values each: halves are exchanged and added, until lane l has
// value l V / 32 (and, of 64, the next one), 32 / V lanes the same one.
template <int V> __device__ __forceinline__ void sums_to_lanes(float (&z)[V], int lane) {
#pragma unroll
    for (int o = 16, have = V; o > 0; o >>= 1) {
        if (have > 1) {
            have /= 2;
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                if (i >= have) break;
                const float give = upper ? z[i] : z[i + have], keep = upper ? z[i + have] : z[i];
                z[i] = keep + __shfl_xor_sync(FULL_MASK, give, o);
            }
        } else {
            z[0] += __shfl_xor_sync(FULL_MASK, z[0], o);
        }
    }
}

// sum += <w, x>, even and odd products in its two halves
template <typename T, int VEC> __device__ __forceinline__ void dot(const Pack<T, VEC> &w, const float (&x)[VEC], float2 &sum) {
    if constexpr (VEC == 1) {
        sum.x = fmaf(to_f32(w.v[0]), x[0], sum.x);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
            sum = fma2(make_float2(to_f32(w.v[i]), to_f32(w.v[i + 1])), make_float2(x[i], x[i + 1]), sum);
    }
}

template <typename T, int N, int VEC>
__global__ void __launch_bounds__(FEW_THREADS, 2)
    k_few_up(const T *__restrict__ x, const T *__restrict__ W, float *__restrict__ m, uint32_t *error, int n, int d, int f) {
    extern __shared__ __align__(32) float few_x[];   // [N][pitch], zeros past n and d
    constexpr int CHUNK = 32 * VEC, ROWS = 2 * UP_UNITS, AHEAD = FEW_AHEAD;
    const int pitch = (d + CHUNK - 1) / CHUNK * CHUNK, lane = threadIdx.x & 31;
    wait_for_prerequisites();
    dependents_may_launch();   // (after the wait: the next kernel reads weights before its own)
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *error = 0;
    x += static_cast<int64_t>(blockIdx.y) * N * d;
    m += static_cast<int64_t>(blockIdx.y) * N * f;
    n = min(n - static_cast<int>(blockIdx.y) * N, N);
    for (int r = threadIdx.x >> 5; r < N; r += FEW_THREADS / 32)
#pragma unroll 4
        for (int c = lane * VEC; c < pitch; c += CHUNK) {   // (d is a multiple of VEC)
            float v[VEC] = {};
            if (r < n && c < d) load_f32<T, VEC>(x + static_cast<int64_t>(r) * d + c, v);
            store_f32<float, VEC>(few_x + r * pitch + c, v);
        }
    __syncthreads();
    const int warps = gridDim.x * (FEW_THREADS / 32);
    for (int j0 = (blockIdx.x * (FEW_THREADS / 32) + (threadIdx.x >> 5)) * UP_UNITS; j0 < f; j0 += warps * UP_UNITS) {
        float2 sum[N * ROWS] = {};   // [row of x][unit][Wg, Wu]
        const T *at[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const int unit = min(j0 + q / 2, f - 1);
            at[q] = W + (static_cast<int64_t>(q % 2 ? f : 0) + unit) * d;
        }
        for (int c0 = lane * VEC; c0 < pitch; c0 += CHUNK * AHEAD) {
            Pack<T, VEC> w[AHEAD][ROWS];
#pragma unroll
            for (int e = 0; e < AHEAD; ++e)
#pragma unroll
                for (int q = 0; q < ROWS; ++q)
                    if (c0 + e * CHUNK < d) w[e][q] = *reinterpret_cast<const Pack<T, VEC> *>(at[q] + c0 + e * CHUNK);
#pragma unroll
            for (int e = 0; e < AHEAD; ++e)
                if (c0 + e * CHUNK < d)
#pragma unroll
                    for (int r = 0; r < N; ++r) {
                        float xv[VEC];
                        load_f32<float, VEC>(few_x + r * pitch + c0 + e * CHUNK, xv);
#pragma unroll
                        for (int q = 0; q < ROWS; ++q) dot<T, VEC>(w[e][q], xv, sum[r * ROWS + q]);
                    }
        }
        constexpr int V = N * ROWS;
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = sum[i].x + sum[i].y;
        sums_to_lanes(acc, lane);
        float a = acc[0], b;
        if constexpr (V == 64) b = acc[1];
        else b = __shfl_xor_sync(FULL_MASK, a, 32 / V);
        const int v = V == 64 ? 2 * lane : lane * V / 32;   // even: this lane has a value of Wg
        const int r = v / ROWS, unit = j0 + v % ROWS / 2;
        if (v % 2 == 0 && (V >= 32 || lane % (32 / V) == 0) && r < n && unit < f)
            m[static_cast<int64_t>(r) * f + unit] = a * sigmoid_of(a) * b;
    }
}

template <typename T, int N, int VEC>
__global__ void __launch_bounds__(FEW_THREADS, 2)
    k_few_down(const float *__restrict__ m, const T *__restrict__ W, T *__restrict__ y, int n, int d, int f) {
    constexpr int CHUNK = 32 * VEC, WARPS = FEW_THREADS / 32, ROWS = DOWN_ROWS, V = N * ROWS;
    __shared__ float share[WARPS][V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j0 = blockIdx.x * ROWS;
    const T *at[ROWS];
#pragma unroll
    for (int q = 0; q < ROWS; ++q) at[q] = W + static_cast<int64_t>(min(j0 + q, d - 1)) * f;
    Pack<T, VEC> w[ROWS];
    int c = warp * CHUNK + lane * VEC;
    auto fetch = [&]() {
#pragma unroll
        for (int q = 0; q < ROWS; ++q)
            if (c < f) w[q] = *reinterpret_cast<const Pack<T, VEC> *>(at[q] + c);
    };
    fetch();   // the kernel before writes no weights, and those before it are done
    wait_for_prerequisites();
    dependents_may_launch();
    m += static_cast<int64_t>(blockIdx.y) * N * f;
    y += static_cast<int64_t>(blockIdx.y) * N * d;
    n = min(n - static_cast<int>(blockIdx.y) * N, N);
    float2 sum[V] = {};   // [row][column of y]
    while (c < f) {
        Pack<T, VEC> now[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) now[q] = w[q];
        const int at_m = c;
        c += WARPS * CHUNK;
        fetch();
#pragma unroll
        for (int r = 0; r < N; ++r)
            if (r < n) {
                float mv[VEC];
                load_f32<float, VEC>(m + static_cast<int64_t>(r) * f + at_m, mv);
#pragma unroll
                for (int q = 0; q < ROWS; ++q) dot<T, VEC>(now[q], mv, sum[r * ROWS + q]);
            }
    }
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = sum[i].x + sum[i].y;
    sums_to_lanes(acc, lane);
    if constexpr (V == 64) {
        share[warp][2 * lane] = acc[0];
        share[warp][2 * lane + 1] = acc[1];
    } else if (lane % (32 / V) == 0) {
        share[warp][lane * V / 32] = acc[0];
    }
    __syncthreads();
    if (threadIdx.x < V) {
        float all = share[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < WARPS; ++k) all += share[k][threadIdx.x];
        const int r = threadIdx.x / ROWS, j = j0 + threadIdx.x % ROWS;
        if (r < n && j < d) y[static_cast<int64_t>(r) * d + j] = from_f32<T>(all);
    }
}

// ---------------------------------------------------------------- host side
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The forms for few rows.  FEW: x has to fit in shared memory.
int few_size(int64_t n) { return n <= 1 ? 1 : n <= 4 ? 4 : FEW_GROUP; }   // rows it is built for
bool few_rows(int64_t n, int64_t d, int dtype) {
    return n <= (dtype == NRNN_F32 ? FEW_MOST : FEW_GROUP) && few_size(n) * (d + 255) * 4 <= static_cast<int64_t>(FEW_X_BYTES);
}
bool short_rows(int64_t n, int64_t d, int64_t f, int dtype, bool aligned) {
    return dtype == NRNN_BF16 && n <= SHORT_MOST && d % 8 == 0 && f % 8 == 0 && aligned;
}

struct Call {
    const void *x, *W_in, *W_out;
    int dtype;
    int64_t n, d, f;
    unsigned char *ws;
    cudaStream_t stream;
};

// Rows up to which bf16 holds m, dL/da and dL/db as two planes, as the form of mma.sync does.
// Roundings of few rows cannot be counted on to average: one of m and one of y leave y up to
// 1.9 times as far off as rounding it once (1 row), 1.52 of 12 rows, under 1.49 from 16 on; two
// planes 1.0.  (8 rows over 1024 x 4096 in a graph: keeping 26.7 -> 28.7 us, backward 41.7 ->
// 49.2; up to 64 rows as much.)
constexpr int TWO_PLANES_MOST = SHORT_MOST;

int inner_planes(int64_t n, int dtype) { return dtype == NRNN_F32 ? 3 : n <= TWO_PLANES_MOST ? 2 : 1; }

// What the gradient takes: p and q, fp32 [2][n][pf] or the blocks of 24 bits, and m
// [planes][n][pf] bf16.
// (Not rounded up, so that its size tells one number of rows from another.)
struct Kept { size_t m, total; int64_t pf; };
Kept kept_layout(int64_t n, int64_t f, int dtype) {
    Kept k{};
    k.pf = ceil_div(f, 8) * 8;
    const size_t planes = inner_planes(n, dtype);
    k.m = dtype == NRNN_BF16 ? ceil_div(n, KEPT_ROWS) * ceil_div(f, KEPT_COLS) * KEPT_BYTES : up256(2 * sizeof(float) * n * k.pf);
    k.total = k.m + 2 * planes * n * k.pf + (planes == 2 ? 24 : 16);
    return k;
}

// The workspace.  An operand of bf16 whose rows are 16-byte aligned is used where it
// lies, every other one is copied to bf16 planes of aligned rows.
struct Plan {
    int planes, inner;   // of x, g and the weights; of m, dL/da and dL/db
    int64_t pd, pf;
    size_t x, w_in, w_out, g, m, gab, parts, total;
};
constexpr size_t NO_COPY = ~static_cast<size_t>(0);

bool used_in_place(const void *p, int64_t row, int dtype) {
    return dtype == NRNN_BF16 && row % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// columns of a tile: equal tiles of whole 64-column blocks, `most` at most
int tile_columns(int64_t N, int most = BN) { return static_cast<int>(ceil_div(ceil_div(N, ceil_div(N, most)), 64) * 64); }

// The same, narrower where tiles are few.  UP and DH: the width that leaves the busiest pair
// the least to do; a tile costs its columns and, for the rows that it reads again, about
// 64 more (UP of 64 rows over 1024 x 4096: 64 tiles of half the width in one wave, 28.7 ->
// 24.6 us forward; of 300 rows they would be two waves, 29.3 -> 36.9).  Tiles that are
// cut: until one is cut in no more than CUT_MOST parts (backward of 1501 x 250 x 683, fp32
// and bf16, at their widest 92 and 54 us, 12 parts 76 and 37, 6 parts 88 and 39; in two, 2000 x
// 512 x 2048 fp32 would go from 192 to 334).
constexpr int CUT_MOST = 12;
int tile_columns_for(int64_t tiles_m, int64_t N, bool cut, int most = BN) {
    int best = most;
    int64_t least = INT64_MAX;
    for (int bn = most; bn >= 64; bn /= 2) {
        const int64_t tiles = tiles_m * ceil_div(N, bn);
        const int64_t load = ceil_div(tiles, PAIRS) * (bn + 64);
        if (!cut && load < least) {
            least = load;
            best = bn;
        }
        if (cut) {
            best = bn;
            if (tiles * CUT_MOST > PAIRS) break;
        }
    }
    return tile_columns(N, best);
}

Plan plan_for(int64_t n, int64_t d, int64_t f, int dtype, bool x_lies, bool w_in_lies, bool w_out_lies, bool g_lies,
              bool keep, bool backward) {
    Plan p{};
    p.planes = dtype == NRNN_F32 ? 3 : 1;
    p.inner = inner_planes(n, dtype);
    p.pd = ceil_div(d, 8) * 8;
    p.pf = ceil_div(f, 8) * 8;
    size_t at = 256;   // the error word
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    p.x = x_lies ? NO_COPY : take(2 * p.planes * n * p.pd);
    p.w_in = w_in_lies ? NO_COPY : take(2 * p.planes * 2 * f * p.pd);
    p.w_out = w_out_lies ? NO_COPY : take(2 * p.planes * d * p.pf);
    p.m = keep || backward ? NO_COPY : take(2 * p.inner * n * p.pf);   // (else among what is kept)
    p.g = !backward || g_lies ? NO_COPY : take(2 * p.planes * n * p.pd);
    p.gab = backward ? take(2 * p.inner * 2 * n * p.pf) : NO_COPY;
    const int64_t widest = tile_columns(d) > tile_columns(f) ? tile_columns(d) : tile_columns(f);
    p.parts = take(sizeof(float) * 2 * PAIRS * BM * widest);
    p.total = at;
    return p;
}

// the operands as bf16 planes: where they lie, or their copies; clears the error word
template <typename T>
cudaError_t operands(const Call &c, const Plan &p, const void *g_in, const void **x, const void **w_in, const void **w_out,
                     const void **g) {
    Copies k{};
    k.error = reinterpret_cast<uint32_t *>(c.ws);
    int64_t rows = 0;
    int n = 0;
    auto take = [&](const void *src, size_t copy, int64_t r, int64_t d, int64_t pitch) -> const void * {
        if (copy == NO_COPY) return src;
        k.src[n] = src;
        k.to[n] = reinterpret_cast<__nv_bfloat16 *>(c.ws + copy);
        k.rows[n] = r;
        k.d[n] = static_cast<int>(d);
        k.pitch[n] = static_cast<int>(pitch);
        rows += r;
        return k.to[n++];
    };
    *x = take(c.x, p.x, c.n, c.d, p.pd);
    *w_in = take(c.W_in, p.w_in, 2 * c.f, c.d, p.pd);
    *w_out = take(c.W_out, p.w_out, c.d, c.f, p.pf);
    if (g != nullptr) *g = take(g_in, p.g, c.n, c.d, p.pd);
    if (rows == 0) return cudaMemsetAsync(k.error, 0, sizeof(uint32_t), c.stream);
    const int64_t b = ceil_div(rows, 8);
    return launch_dependent(k_planes<T>, static_cast<unsigned>(b < 4864 ? b : 4864), 256, 0, c.stream, k);
}

template <int FORM, typename T, bool KEEP = false>
cudaError_t gemm(const Call &c, const CUtensorMap &tmA, const CUtensorMap &tmB, const CUtensorMap &tmOut, GemmArgs a) {
    static std::atomic<unsigned long long> configured{0};
    constexpr size_t smem = gemm_smem<FORM, T>();
    cudaError_t e = once_per_device(configured, [](int) {
        return cudaFuncSetAttribute(k_mlp_gemm<FORM, T, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    });
    if (e != cudaSuccess) return e;
    const int64_t tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
    const int64_t most = CUTS<FORM> ? tiles * a.kb : tiles;
    if (most > INT32_MAX) return cudaErrorInvalidConfiguration;
    const int pairs = static_cast<int>(most < PAIRS ? most : PAIRS);
    a.side = 1;
    a.teams = pairs;
    a.units = a.whole = static_cast<int>(tiles);
    if (CUTS<FORM>) {
        // teams of pairs with the column tiles of one row tile side by side
        a.side = a.tiles_n <= MOST_SIDE && a.tiles_n <= pairs ? a.tiles_n : 1;
        a.teams = pairs / a.side;
        a.units = static_cast<int>(tiles / a.side);
        a.whole = a.units >= WAVES_UNCUT * a.teams ? a.units : a.units / a.teams * a.teams;
        const int slices = (a.units - a.whole) * a.kb;   // (fits: `most` does)
        a.share = slices / a.teams;
        a.longer = slices % a.teams;
    }
    e = launch_dependent(k_mlp_gemm<FORM, T, KEEP>, 2 * pairs, GEMM_THREADS, smem, c.stream, tmA, tmB, tmOut, a);
    const int64_t cut = static_cast<int64_t>(a.units - a.whole) * a.side;
    if (e == cudaSuccess && cut > 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cut), BM / JOIN_ROWS);
        cfg.blockDim = dim3(JOIN_THREADS);
        cfg.stream = c.stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, k_join_parts<FORM, T>, a);
    }
    return e;
}

// a map over bf16 (planes, rows, inner) whose rows are pitch elements apart
bool map(CUtensorMap *m, const void *base, int64_t inner, int64_t pitch, int64_t rows, int64_t planes, int box_inner, int box_rows) {
    return make_map_pitched(m, base, inner, pitch, rows, planes, box_inner, box_rows);
}

GemmArgs args_of(const Call &c, const Plan &p, int64_t M, int64_t N, int64_t K, int bn) {
    GemmArgs a{};
    a.error = reinterpret_cast<uint32_t *>(c.ws);
    a.wait_ns = wait_limit_ns();
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.bn = bn;
    a.tiles_m = static_cast<int>(ceil_div(M, BM));
    a.tiles_n = static_cast<int>(ceil_div(N, bn));
    a.kb = static_cast<int>(ceil_div(K, BK));
    a.kept_cols = static_cast<int>(ceil_div(c.f, KEPT_COLS));
    a.inner = p.inner;
    return a;
}

template <typename T> int forward(const Call &c, const Plan &p, T *y, unsigned char *kept) {
    unsigned char *m = kept != nullptr ? kept + kept_layout(c.n, c.f, c.dtype).m : c.ws + p.m;
    const void *x, *w_in, *w_out;
    if (operands<T>(c, p, nullptr, &x, &w_in, &w_out, nullptr) != cudaSuccess) return NRNN_ERR_CUDA;
    CUtensorMap ta, tb, to;
    const int units = tile_columns_for(ceil_div(c.n, BM), c.f, false, BN / 2);   // UP: a tile's units
    if (!map(&ta, x, c.d, p.pd, c.n, p.planes, BK, HALF_M) || !map(&tb, w_in, c.d, p.pd, c.f, 2 * p.planes, BK, units) ||
        !map(&to, m, c.f, p.pf, c.n, p.inner, PIECE, BOX_ROWS))
        return NRNN_ERR_CUDA;
    GemmArgs a = args_of(c, p, c.n, c.f, c.d, 2 * units);
    a.tiles_n = static_cast<int>(ceil_div(c.f, units));
    a.pq = kept;
    a.pitch = static_cast<int>(p.pf);
    if ((kept != nullptr ? gemm<UP, T, true>(c, ta, tb, to, a) : gemm<UP, T>(c, ta, tb, to, a)) != cudaSuccess) return NRNN_ERR_CUDA;
    const int bn = tile_columns_for(ceil_div(c.n, BM), c.d, true);
    a = args_of(c, p, c.n, c.d, c.f, bn);
    a.parts = reinterpret_cast<float *>(c.ws + p.parts);
    a.out = y;
    a.blocks_out = used_in_place(y, c.d, c.dtype);
    if (!map(&ta, m, c.f, p.pf, c.n, p.inner, BK, HALF_M) || !map(&tb, w_out, c.f, p.pf, c.d, p.planes, BK, bn / 2) ||
        (a.blocks_out && !map(&to, y, c.d, c.d, c.n, 1, PIECE, BOX_ROWS)))
        return NRNN_ERR_CUDA;
    return gemm<DOWN, T>(c, ta, tb, to, a) == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

template <typename T>
int backward(const Call &c, const Plan &p, const unsigned char *kept, const void *g_, T *gx, T *gW_in, T *gW_out) {
    const Kept kl = kept_layout(c.n, c.f, c.dtype);
    const unsigned char *m = kept + kl.m;
    unsigned char *gab = c.ws + p.gab;
    const void *x, *w_in, *w_out, *g;
    if (operands<T>(c, p, g_, &x, &w_in, &w_out, &g) != cudaSuccess) return NRNN_ERR_CUDA;
    CUtensorMap ta, tb, to;
    float *parts = reinterpret_cast<float *>(c.ws + p.parts);
    // fp32: one piece of an epilogue warp holds ga and gb, so tiles of 128
    int bn = tile_columns_for(ceil_div(c.n, BM), c.f, false, p.planes != 1 ? 2 * PIECE : BN);
    GemmArgs a = args_of(c, p, c.n, c.f, c.d, bn);
    a.pq = const_cast<unsigned char *>(kept);
    a.pitch = static_cast<int>(p.pf);
    if (!map(&ta, g, c.d, p.pd, c.n, p.planes, BK, HALF_M) || !map(&tb, w_out, c.f, p.pf, c.d, p.planes, 64, BK) ||
        !map(&to, gab, c.f, p.pf, c.n, 2 * p.inner, PIECE, BOX_ROWS))
        return NRNN_ERR_CUDA;
    if (gemm<DH, T>(c, ta, tb, to, a) != cudaSuccess) return NRNN_ERR_CUDA;
    // gx
    bn = tile_columns_for(ceil_div(c.n, BM), c.d, true);
    a = args_of(c, p, c.n, c.d, c.f, bn);
    a.kb_half = a.kb;
    a.kb *= 2;
    a.parts = parts;
    a.out = gx;
    a.blocks_out = used_in_place(gx, c.d, c.dtype);
    if (!map(&ta, gab, c.f, p.pf, c.n, 2 * p.inner, BK, HALF_M) || !map(&tb, w_in, c.d, p.pd, c.f, 2 * p.planes, 64, BK) ||
        (a.blocks_out && !map(&to, gx, c.d, c.d, c.n, 1, PIECE, BOX_ROWS)))
        return NRNN_ERR_CUDA;
    if (gemm<GX, T>(c, ta, tb, to, a) != cudaSuccess) return NRNN_ERR_CUDA;
    // gW_in
    bn = tile_columns_for(2 * ceil_div(c.f, BM), c.d, true);
    a = args_of(c, p, c.f, c.d, c.n, bn);
    a.m_half = a.tiles_m;
    a.tiles_m *= 2;
    a.parts = parts;
    a.out = gW_in;
    a.blocks_out = used_in_place(gW_in, c.d, c.dtype);
    if (!map(&ta, gab, c.f, p.pf, c.n, 2 * p.inner, 64, BK) || !map(&tb, x, c.d, p.pd, c.n, p.planes, 64, BK) ||
        (a.blocks_out && !map(&to, gW_in, c.d, c.d, c.f, 2, PIECE, BOX_ROWS)))
        return NRNN_ERR_CUDA;
    if (gemm<GWI, T>(c, ta, tb, to, a) != cudaSuccess) return NRNN_ERR_CUDA;
    // gW_out
    bn = tile_columns_for(ceil_div(c.d, BM), c.f, true);
    a = args_of(c, p, c.d, c.f, c.n, bn);
    a.parts = parts;
    a.out = gW_out;
    a.blocks_out = used_in_place(gW_out, c.f, c.dtype);
    if (!map(&ta, g, c.d, p.pd, c.n, p.planes, 64, BK) || !map(&tb, m, c.f, p.pf, c.n, p.inner, 64, BK) ||
        (a.blocks_out && !map(&to, gW_out, c.f, c.f, c.d, 1, PIECE, BOX_ROWS)))
        return NRNN_ERR_CUDA;
    return gemm<GWO, T>(c, ta, tb, to, a) == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

template <typename T, int N, int VEC_UP, int VEC_DOWN>
cudaError_t launch_few(const Call &c, T *y) {
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = once_per_device(configured, [](int) {
        return cudaFuncSetAttribute(k_few_up<T, N, VEC_UP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(FEW_X_BYTES));
    });
    if (e != cudaSuccess) return e;
    float *m = reinterpret_cast<float *>(c.ws + 256);
    const int n = static_cast<int>(c.n), d = static_cast<int>(c.d), f = static_cast<int>(c.f);
    const size_t smem = sizeof(float) * N * (ceil_div(d, 32 * VEC_UP) * 32 * VEC_UP);
    const int64_t want = ceil_div(f, UP_UNITS * (FEW_THREADS / 32));
    const unsigned groups = static_cast<unsigned>(ceil_div(n, N));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < 304 ? want : 304), groups);
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_few_up<T, N, VEC_UP>, static_cast<const T *>(c.x), static_cast<const T *>(c.W_in), m,
                           reinterpret_cast<uint32_t *>(c.ws), n, d, f);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(d, DOWN_ROWS)), groups);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k_few_down<T, N, VEC_DOWN>, static_cast<const float *>(m), static_cast<const T *>(c.W_out), y,
                              n, d, f);
}

template <typename T, int N> cudaError_t launch_few(const Call &c, T *y) {
    constexpr int WIDE = 16 / sizeof(T);
    const bool up = c.d % WIDE == 0 && (reinterpret_cast<uintptr_t>(c.W_in) | reinterpret_cast<uintptr_t>(c.x)) % 16 == 0;
    const bool down = c.f % WIDE == 0 && reinterpret_cast<uintptr_t>(c.W_out) % 16 == 0;
    if constexpr (sizeof(T) == 4)   // (bf16 that is aligned throughout takes the mma.sync form)
        if (up && down) return launch_few<T, N, WIDE, WIDE>(c, y);
    return up     ? launch_few<T, N, WIDE, 1>(c, y)
           : down ? launch_few<T, N, 1, WIDE>(c, y)
                  : launch_few<T, N, 1, 1>(c, y);
}

template <typename T> int few_forward(const Call &c, T *y) {
    cudaError_t e;
    switch (few_size(c.n)) {
        case 1: e = launch_few<T, 1>(c, y); break;
        case 4: e = launch_few<T, 4>(c, y); break;
        default: e = launch_few<T, FEW_GROUP>(c, y);
    }
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

template <int TILES> cudaError_t launch_short(const Call &c, void *y) {
    __nv_bfloat16 *m = reinterpret_cast<__nv_bfloat16 *>(c.ws + 256);
    const int n = static_cast<int>(c.n), d = static_cast<int>(c.d), f = static_cast<int>(c.f);
    const cudaError_t e = launch_dependent(k_short_up<TILES>, static_cast<unsigned>(ceil_div(f, 8)), UP_WARPS * 32, 0, c.stream,
                                           static_cast<const __nv_bfloat16 *>(c.x), static_cast<const __nv_bfloat16 *>(c.W_in), m,
                                           reinterpret_cast<uint32_t *>(c.ws), n, d, f);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_short_down<TILES>, static_cast<unsigned>(ceil_div(d, 16)), DOWN_WARPS * 32, 0, c.stream,
                            static_cast<const __nv_bfloat16 *>(m), static_cast<const __nv_bfloat16 *>(c.W_out),
                            static_cast<__nv_bfloat16 *>(y), n, d, f);
}

int short_forward(const Call &c, void *y) {
    const cudaError_t e = c.n <= 8 ? launch_short<1>(c, y) : launch_short<2>(c, y);
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

// nothing kept: the workspace of the forms for few rows, the error word and m
size_t few_bytes(int64_t n, int64_t f) { return up256(256 + sizeof(float) * n * f); }

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
    return kept_layout(rows, f, dtype).total;
}

size_t nrnn_gated_mlp_workspace_bytes(int64_t rows, int64_t d, int64_t f, int dtype, int what) {
    if (d <= 0 || what < 0 || what > 2 || !sizes_fit(0, d, 1) || nrnn_gated_mlp_kept_bytes(rows, f, dtype) == 0) return 0;
    // nothing kept: enough for whichever form the call takes (an unaligned tensor's may be another)
    if (what == 0 && few_rows(rows, d, dtype)) return few_bytes(rows, f);
    return plan_for(rows, d, f, dtype, false, false, false, false, what == 2, what == 1).total;
}

int nrnn_gated_mlp_forward(const void *x, const void *W_in, const void *W_out, int dtype, int64_t rows, int64_t d,
                           int64_t f, void *y, void *kept, void *workspace, size_t ws_bytes, void *stream) {
    const Call c{x, W_in, W_out, dtype, rows, d, f, static_cast<unsigned char *>(workspace), static_cast<cudaStream_t>(stream)};
    const int st = check(c);
    if (st != NRNN_OK) return st;
    if (rows == 0) return NRNN_OK;
    const uintptr_t elem = dtype == NRNN_BF16 ? 2 : 4;
    const int64_t xb = rows * d * elem, wb = f * d * elem;
    if (y == nullptr || reinterpret_cast<uintptr_t>(y) % elem != 0 || reinterpret_cast<uintptr_t>(kept) % 256 != 0 ||
        !outputs_apart({{y, xb}, {kept, static_cast<int64_t>(nrnn_gated_mlp_kept_bytes(rows, f, dtype))}},
                       {{x, xb}, {W_in, 2 * wb}, {W_out, wb}}))
        return NRNN_ERR_INVALID_ARG;
    if (kept == nullptr) {
        const bool aligned = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(W_in) |
                               reinterpret_cast<uintptr_t>(W_out)) & 15) == 0;
        const bool in_short = short_rows(rows, d, f, dtype, aligned);
        if (in_short || few_rows(rows, d, dtype)) {
            if (!usable(workspace, ws_bytes, few_bytes(rows, f))) return NRNN_ERR_WORKSPACE;
            return in_short ? short_forward(c, y)
                 : dtype == NRNN_BF16 ? few_forward(c, static_cast<__nv_bfloat16 *>(y)) : few_forward(c, static_cast<float *>(y));
        }
    }
    const Plan p = plan_for(rows, d, f, dtype, used_in_place(x, d, dtype), used_in_place(W_in, d, dtype),
                            used_in_place(W_out, f, dtype), false, kept != nullptr, false);
    if (!usable(workspace, ws_bytes, p.total)) return NRNN_ERR_WORKSPACE;
    unsigned char *k = static_cast<unsigned char *>(kept);
    return dtype == NRNN_BF16 ? forward(c, p, static_cast<__nv_bfloat16 *>(y), k) : forward(c, p, static_cast<float *>(y), k);
}

int nrnn_gated_mlp_backward(const void *x, const void *W_in, const void *W_out, const void *kept, const void *g,
                            int dtype, int64_t rows, int64_t d, int64_t f, void *gx, void *gW_in, void *gW_out,
                            void *workspace, size_t ws_bytes, void *stream) {
    const Call c{x, W_in, W_out, dtype, rows, d, f, static_cast<unsigned char *>(workspace), static_cast<cudaStream_t>(stream)};
    const int st = check(c);
    if (st != NRNN_OK) return st;
    const uintptr_t elem = dtype == NRNN_BF16 ? 2 : 4;
    const int64_t xb = rows * d * elem, wb = f * d * elem;
    if (gW_in == nullptr || gW_out == nullptr ||
        (rows > 0 && (g == nullptr || gx == nullptr || kept == nullptr || reinterpret_cast<uintptr_t>(kept) % 256 != 0)) ||
        (reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(gx) | reinterpret_cast<uintptr_t>(gW_in) |
         reinterpret_cast<uintptr_t>(gW_out)) % elem != 0 ||
        !outputs_apart({{gx, xb}, {gW_in, 2 * wb}, {gW_out, wb}},
                       {{x, xb}, {W_in, 2 * wb}, {W_out, wb}, {g, xb},
                        {kept, static_cast<int64_t>(nrnn_gated_mlp_kept_bytes(rows, f, dtype))}}))
        return NRNN_ERR_INVALID_ARG;
    if (rows == 0)
        return cudaMemsetAsync(gW_in, 0, elem * 2 * f * d, c.stream) == cudaSuccess &&
                       cudaMemsetAsync(gW_out, 0, elem * f * d, c.stream) == cudaSuccess
                   ? NRNN_OK : NRNN_ERR_CUDA;
    const Plan p = plan_for(rows, d, f, dtype, used_in_place(x, d, dtype), used_in_place(W_in, d, dtype),
                            used_in_place(W_out, f, dtype), used_in_place(g, d, dtype), true, true);
    if (!usable(workspace, ws_bytes, p.total)) return NRNN_ERR_WORKSPACE;
    const unsigned char *k = static_cast<const unsigned char *>(kept);
    return dtype == NRNN_BF16
               ? backward(c, p, k, g, static_cast<__nv_bfloat16 *>(gx), static_cast<__nv_bfloat16 *>(gW_in),
                          static_cast<__nv_bfloat16 *>(gW_out))
               : backward(c, p, k, g, static_cast<float *>(gx), static_cast<float *>(gW_in), static_cast<float *>(gW_out));
}

}  // extern "C"
