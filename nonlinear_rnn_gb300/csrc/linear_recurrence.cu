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
// r and i are bounded below by 2^-63 (the exponential is clamped, so that two sigmoids
// share a reciprocal and 1 - r is exact to rounding on both sides); where s is zero all
// the same (1 - a^2 below 2^-126, which the square root takes for zero) the term with a^2 / s
// is left out, which is its limit as r vanishes.
//
// One pass over the data in each direction, bound by HBM: 4 values a unit and step
// forward, 8 backward.  A tile is 64 units (two a lane, on packed f32x2 arithmetic) and
// SEG steps a warp; TMA brings it to shared memory and takes the result from there.
// CTAs are persistent: they take tiles from a counter, every column's next chunk after
// all columns' chunks before it (backward: from the end of time), and start the copies
// of the next tile while they work on one.  A thread composes the maps h -> A h + B of
// its steps, the warps' maps meet in shared memory, and the carry into the chunk comes
// from a look-back whose grouping is fixed: chunks form groups of `group`, groups form
// spans of `span`.  A chunk publishes its map, and a group's last chunk that of the group.
// A chunk folds, in order, the maps of its span's groups and of its group's chunks before
// it, and starts them from the state at the end of the span before, which that span's
// last chunk publishes.  So no result depends on timing, and a chain has one hop a span.
//
// A sequence's first state (backward: the gradient of its last) cuts the scan: the map
// of a step that begins a pack's segment is marked by the sign of its A (a decay is
// never negative), and what a marked map is applied to is not looked at, NaN or not.
//
// A pack of enough segments is cut into chunks of each segment instead of chunks of the
// time axis (the plan of pack_plan.cuh, built beside the clearing of the slots): then
// every segment is a column of its own, and many chains are short instead of few long.
// A segment's short last chunk loads steps of the next one, which it leaves out, and
// stores its own by rows.  (262144 x 512 fp32 in 64 segments, backward: 952 -> 807 us.)
// Where one segment is so long that its chain would be what takes the time, which only the
// device knows, the same kernel goes by the time axis (by_segments).
//
// Measured, with HBM's measured copy rate of 6775 GB/s: 16 x 16384 x 1024 bf16 395 us forward
// (0.80), 720 backward (0.88); 4 x 131072 x 64 fp32 143 us (0.55: four columns; without the
// look-back 0.96); the pack 744 us backward (0.85).  Timing-only copies of the forward
// without the look-back take 345 us: the rest is issue slots (62% busy, 16 warps an SM; two
// values of every step are held in registers between the scan's two halves).
//
// A wait that gives up (the limit of nrnn_set_wait_limit_ns) sets the workspace's second
// word, which ends the other waits too, and gives NaN in what depended on it.
#include <type_traits>

#include "../../include/nrnn.h"
#include "nrnn_device.cuh"
#include "nrnn_internal.h"
#include "pack_plan.cuh"
#include "rows.cuh"
#include "tcgen05.cuh"

namespace nrnn {
namespace {

constexpr int UNITS = 64, NW = 4, THREADS = NW * 32;
constexpr uint64_t SETTLE_NS = 2000000000ull;   // for copies in flight after a wait gave up

// A kernel's form.  WIDE: many columns, so few chunks of one are under way at a time:
// tickets and copies run a tile ahead, and every warp reads the few maps before by
// itself.  Else chunks of a column wait for many others: tickets are taken late, and the
// warps share the maps before.
// MODE: how sequences lie.  ROWS: the rows of a batch; PACK: a pack cut by time; PLAN: a
// pack cut by segments (a WIDE form).
enum Mode { ROWS, PACK, PLAN };

template <typename TS, bool WIDE> struct Shape {
    static constexpr int SEG = sizeof(TS) == 2 ? 16 : 8;      // steps a warp
    static constexpr int L = NW * SEG, PLANE = L * UNITS;     // steps and elements of a tile's block
    static constexpr int FORWARD_CTAS = WIDE || sizeof(TS) == 2 ? 4 : 5, BACKWARD_CTAS = 4;   // an SM
    static constexpr int FORWARD_TILES = WIDE ? 2 : 1;        // in shared memory
};

struct RecArgs {
    const void *H;                    // backward: (B, T, d)
    void *H_out, *gP;                 // PLAN: short chunks are stored by rows
    const float *params, *state;      // (3, d); (rows, d) or null
    const int32_t *cu;                // pack: (rows + 1) offsets
    int rows;                         // sequences: B or segments
    int T, d;
    int n_ut, n_cols, n_chunks;       // unit tiles; B n_ut; chunks of time
    int group, span;                  // look-back: chunks of a group, groups of a span
    uint32_t n_tiles;
    float *last;                      // forward: (rows, d) or null
    const float *g_last;              // backward: (rows, d) or null
    float *g_state;                   // backward: (rows, d) or null
    float *part;                      // backward: [n_cols][n_chunks][3][UNITS] sums of a tile
    const int4 *plan;                 // PLAN: the chunks after plan[0] = {how many, whether the call goes by
                                      // them}; n_chunks is their most, n_cols the unit tiles
    unsigned long long *slots;        // [n_cols][n_chunks][UNITS] maps of chunks (WIDE: of a group's last
                                      // chunk the state after it)
    unsigned long long *maps;         // [n_cols][groups][UNITS] maps of groups
    unsigned long long *ends;         // [n_cols][spans][UNITS] states after a span
    uint32_t *ticket;
    uint32_t *error;
    uint64_t wait_ns;
};

// ---------------------------------------------------------------- the gates
struct UnitWeights {   // of a lane's two units
    float2 fall2, nb_a, nb_i;   // -rate log2 e; -b log2 e
};

__device__ __forceinline__ float2 two_of(const float *p, bool ok) {
    return ok ? *reinterpret_cast<const float2 *>(p) : make_float2(0.f, 0.f);
}
__device__ __forceinline__ UnitWeights weights_of(const float *params, int d, int u, bool ok) {
    UnitWeights w;
    w.fall2 = mul2(two_of(params + u, ok), splat2(-LOG2E));
    w.nb_a = mul2(two_of(params + d + u, ok), splat2(-LOG2E));
    w.nb_i = mul2(two_of(params + 2 * d + u, ok), splat2(-LOG2E));
    return w;
}

__device__ __forceinline__ float2 load2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *p) {
    const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / sqrt(x); 0 below 2^-126, where sqrt_approx is 0 (and where rsqrt would be infinite)
__device__ __forceinline__ float rsqrt_or_zero(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return x >= 1.17549435e-38f ? y : 0.f;
}

// The decay a = 2^z, z <= 0, near one: a - 1 by its series (ex2.approx is 2^-22 off, to one
// side over a range, and a unit of long memory adds that up; one more than the series is a
// rounding of 2^-25 off), and a^2 - 1 = (a - 1)(a + 1) without a difference.  Beyond the
// border a^2 - 1 is a difference, and ex2's error in it grows by 2 a^2 / (1 - a^2).
// TERMS 5: to z = -0.18, where that leaves s 2^-20 off at most; 3: to -0.045, 2^-18 (measured
// beside the borders: 3.3e-7 and 1.3e-6, on the series' side 1.6e-7).  The forward takes 5
// whatever the storage, as its last states are fp32 and go on in steps (16 x 16384 x 1024 bf16
// 392 us with 3, 396 with 5); the backward of bf16 takes 3 (711 us, 731).
template <int TERMS> struct NearOne {
    static constexpr float LIMIT = TERMS == 5 ? -0.18f : -0.045f;
    __device__ static float2 less_one(float2 z) {
        constexpr float C1 = 0.6931471806f, C2 = 0.2402265070f, C3 = 0.0555041087f, C4 = 0.0096181291f, C5 = 0.0013333558f,
                        C6 = 0.0001540353f;   // (ln 2)^k / k!
        float2 p = TERMS == 5 ? fma2(z, splat2(C6), splat2(C5)) : splat2(C4);
        if (TERMS == 5) p = fma2(z, p, splat2(C4));
        p = fma2(z, p, splat2(C3));
        p = fma2(z, p, splat2(C2));
        p = fma2(z, p, splat2(C1));
        return mul2(z, p);
    }
};
template <int TERMS> __device__ __forceinline__ float2 decay_of(float2 z) {
    const float2 one_more = add2(NearOne<TERMS>::less_one(z), splat2(1.f)), far = ex2_2(z);
    return make_float2(z.x > NearOne<TERMS>::LIMIT ? one_more.x : far.x, z.y > NearOne<TERMS>::LIMIT ? one_more.y : far.y);
}
// the decay, and a^2 - 1
template <int TERMS> __device__ __forceinline__ float2 decay_of(float2 z, float2 &square_less_one) {
    const float2 e = NearOne<TERMS>::less_one(z), one_more = add2(e, splat2(1.f)), q = mul2(e, add2(e, splat2(2.f)));
    const float2 far = ex2_2(z), far_q = fma2(far, far, splat2(-1.f));
    const bool x = z.x > NearOne<TERMS>::LIMIT, y = z.y > NearOne<TERMS>::LIMIT;
    square_less_one = make_float2(x ? q.x : far_q.x, y ? q.y : far_q.y);
    return make_float2(x ? one_more.x : far.x, y ? one_more.y : far.y);
}

// e^-x in exponent-2 units, clamped: 1 / (1 + e) = sig, e / (1 + e) = 1 - sig
__device__ __forceinline__ float2 falling(float2 p, float2 nb) {
    return ex2_2(clamp2(fma2(p, splat2(-LOG2E), nb)));
}

template <int TERMS>
__device__ __forceinline__ void forward_gates(float2 pa, float2 pi, float2 v, const UnitWeights &w, float2 &a, float2 &u) {
    const float2 one = splat2(1.f);
    const float2 da = add2(falling(pa, w.nb_a), one), di = add2(falling(pi, w.nb_i), one);
    const float2 inv = rcp_2(mul2(da, di));
    const float2 r = mul2(inv, di), i = mul2(inv, da);
    const float2 z = mul2(w.fall2, r);
    float2 q;
    a = decay_of<TERMS>(z, q);
    u = mul2(mul2(make_float2(sqrt_approx(-q.x), sqrt_approx(-q.y)), i), v);
}


// ------------------------------------------------------ maps h -> A h + B of two units
struct Map2 { float2 A, B; };

__device__ __forceinline__ bool marked(float A) { return __float_as_int(A) < 0; }
template <bool CUTS> __device__ __forceinline__ float apply(float A, float B, float h) {
    const float y = fmaf(A, h, B);
    return CUTS && marked(A) ? B : y;
}
template <bool CUTS> __device__ __forceinline__ float2 apply(const Map2 &m, float2 h) {
    if (!CUTS) return fma2(m.A, h, m.B);
    return make_float2(apply<true>(m.A.x, m.B.x, h.x), apply<true>(m.A.y, m.B.y, h.y));
}
__device__ __forceinline__ float both(float A1, float A2) {   // the product, marked if either is
    return __uint_as_float(__float_as_uint(A1 * A2) | ((__float_as_uint(A1) | __float_as_uint(A2)) & 0x80000000u));
}
// m1, then m2
template <bool CUTS> __device__ __forceinline__ Map2 then(const Map2 &m1, const Map2 &m2) {
    Map2 m;
    m.B = apply<CUTS>(m2, m1.B);
    m.A = CUTS ? make_float2(both(m1.A.x, m2.A.x), both(m1.A.y, m2.A.y)) : mul2(m1.A, m2.A);
    return m;
}

// a lane's two slots; the pair of either is its own ready flag (see publish)
__device__ __forceinline__ void publish2(unsigned long long *slot, const Map2 &m) {
    unsigned long long v0 = pack_pair(m.A.x, m.B.x), v1 = pack_pair(m.A.y, m.B.y);
    if (v0 == SLOT_EMPTY) v0 = pack_pair(0.f, -0.f);
    if (v1 == SLOT_EMPTY) v1 = pack_pair(0.f, -0.f);
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(slot), "l"(v0), "l"(v1) : "memory");
}
__device__ __forceinline__ ulonglong2 peek2(const unsigned long long *slot) {
    ulonglong2 v;
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "l"(slot) : "memory");
    return v;
}
__device__ __forceinline__ bool there(const ulonglong2 &v) { return v.x != SLOT_EMPTY && v.y != SLOT_EMPTY; }
__device__ __forceinline__ Map2 map_of(const ulonglong2 &v) {
    return Map2{make_float2(pair_A(v.x), pair_A(v.y)), make_float2(pair_b(v.x), pair_b(v.y))};
}
// waits for a slot; a map of NaN if it gave up or another wait of the call did
__device__ __forceinline__ Map2 await2(const unsigned long long *slot, ulonglong2 v, const RecArgs &a) {
    if (!there(v)) {
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            v = peek2(slot);
            if (there(v)) break;
            __nanosleep(32);
            const bool late = globaltimer_ns() - t0 > a.wait_ns;
            if (late) atomicOr(a.error, 1u);
            if (late || *static_cast<volatile uint32_t *>(a.error) != 0) {
                const float nan = __int_as_float(0x7fffffff);
                return Map2{splat2(nan), splat2(nan)};
            }
        }
    }
    return map_of(v);
}

// What a CTA shares while it works on a tile
struct Shared {
    float2 aggA[2][NW][32], aggB[2][NW][32];   // maps of the warps' steps, in the scan's order
    float2 preA[NW][32], preB[NW][32];         // maps of runs of groups (0, 1) and chunks (2, 3) before
    float2 end[32];                            // state after the span before
    uint64_t bar[2];
    uint32_t tile[2];
};

// Chunks of a group where columns are many (spans of one group).  A chain has a hop a
// group, about 1.3 us, which a chunk's longer work hides backward.  (16 x 16384 x 1024 bf16
// forward in groups of 2, 4, 8: 386, 391, 402 us, but 8 x 32768: 562, 505 for 2, 4; backward
// 717, 771, 975, and 847, 832.)
template <bool REVERSE> constexpr int WIDE_GROUP = REVERSE ? 2 : 4;

// Where a tile lies: row, first unit, chunk q of nq in the scan's order, its steps t0 .. (of a
// sequence that ends before t_end), and its place among all chunks (slots, sums)
struct Place { int col, b, u0, q, nq, t0, t_end; int64_t at; };
template <int L, bool REVERSE, int MODE> __device__ __forceinline__ Place place_of(const RecArgs &a, uint32_t tile) {
    Place p;
    if constexpr (MODE == PLAN) {
        const int item = static_cast<int>(tile / static_cast<uint32_t>(a.n_ut)), ut = static_cast<int>(tile) - item * a.n_ut;
        const int4 e = a.plan[1 + item];   // first step, the segment's end, chunk j of it, place among all chunks
        const int after = (e.y - e.x + L - 1) / L;   // chunks from this one on
        p.col = ut;
        p.b = 0;
        p.u0 = ut * UNITS;
        p.nq = e.z + after;
        p.q = REVERSE ? after - 1 : e.z;
        p.t0 = e.x;
        p.t_end = e.y;
        p.at = static_cast<int64_t>(ut) * a.n_chunks + (e.w - e.z) + p.q;
        return p;
    }
    p.q = static_cast<int>(tile / static_cast<uint32_t>(a.n_cols));
    p.col = static_cast<int>(tile) - p.q * a.n_cols;
    p.b = p.col / a.n_ut;
    p.u0 = (p.col - p.b * a.n_ut) * UNITS;
    p.nq = a.n_chunks;
    p.t0 = (REVERSE ? a.n_chunks - 1 - p.q : p.q) * L;
    p.t_end = a.T;
    p.at = static_cast<int64_t>(p.col) * a.n_chunks + p.q;
    return p;
}
// whether a call with a plan goes by its segments (k_prepare decides)
__device__ __forceinline__ bool by_segments(const int4 *plan) { return plan[0].y != 0; }
// tiles there are
template <int MODE> __device__ __forceinline__ uint32_t tiles_of(const RecArgs &a) {
    return MODE == PLAN ? static_cast<uint32_t>(a.plan[0].x) * a.n_ut : a.n_tiles;
}
// the segment of a step
__device__ __forceinline__ int segment_of(const RecArgs &a, int t) {
    int lo = 0, hi = a.rows;   // the last seg with cu[seg] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The carry into this warp's steps.  it: the CTA's count of tiles; p: its tile (q: the
// chunk in the scan's order, backward from the end of time); m: the map of this warp's
// steps; place: the warp in the scan's order; first: the state that the first span starts
// from; ok: the tile's copies came.  Called by all threads; between() runs after the last
// barrier.
template <bool WIDE, bool REVERSE, bool CUTS, typename Fn>
__device__ __forceinline__ float2 carry_into(const RecArgs &a, Shared &s, int it, const Place &p, int place, int lane,
                                             const Map2 &m, float2 first, bool ok, Fn &&between) {
    constexpr int GROUP = WIDE_GROUP<REVERSE>;
    const int q = p.q;
    const float2 nan = splat2(__int_as_float(0x7fffffff));
    float2 (&aggA)[NW][32] = s.aggA[it & 1], (&aggB)[NW][32] = s.aggB[it & 1];
    aggA[place][lane] = m.A;
    aggB[place][lane] = ok ? m.B : nan;   // (a tile whose copies gave up)
    auto warps_map = [&](int w) { return Map2{aggA[w][lane], aggB[w][lane]}; };
    auto whole_tile = [&]() {
        Map2 all = warps_map(0);
#pragma unroll
        for (int w = 1; w < NW; ++w) all = then<CUTS>(all, warps_map(w));
        return all;
    };
    unsigned long long *const slot = a.slots + p.at * UNITS + 2 * lane;
    float2 h = first;
    if constexpr (WIDE) {
        const int g = q / GROUP, before = q % GROUP;
        const bool closes = before + 1 == GROUP && q + 1 < p.nq;
        const unsigned long long *const end = slot - (before + 1) * UNITS;   // the state after the group before
        ulonglong2 v[GROUP - 1], e = make_ulonglong2(SLOT_EMPTY, SLOT_EMPTY);
        if (g > 0) e = peek2(end);
#pragma unroll
        for (int k = 1; k < GROUP; ++k)   // chunk q - k
            if (k <= before) v[k - 1] = peek2(slot - k * UNITS);
        __syncthreads();
        between();
        if (place == 0 && !closes) publish2(slot, whole_tile());
        if (g > 0) h = await2(end, e, a).B;
#pragma unroll
        for (int k = GROUP - 1; k > 0; --k)
            if (k <= before) h = apply<CUTS>(await2(slot - k * UNITS, v[k - 1], a), h);
        if (!ok) h = nan;
        if (place == 0 && closes) publish2(slot, Map2{splat2(0.f), apply<CUTS>(whole_tile(), h)});
    } else {
        const int g = q / a.group, before = q - g * a.group, sp = g / a.span, gi = g - sp * a.span;
        const int groups = (a.n_chunks + a.group - 1) / a.group, spans = (groups + a.span - 1) / a.span;
        unsigned long long *const map = a.maps + (static_cast<int64_t>(p.col) * groups + g) * UNITS + 2 * lane;
        unsigned long long *const end = a.ends + (static_cast<int64_t>(p.col) * spans + sp) * UNITS + 2 * lane;
        const bool closes = before + 1 == a.group, closes_span = closes && gi + 1 == a.span;
        __syncthreads();
        Map2 all{};
        if (place == 0) {
            all = whole_tile();
            if (!closes) publish2(slot, all);
        }
        // maps before: the first two warps take halves of the span's groups, the others
        // of the group's chunks
        const unsigned long long *const list =
            place < 2 ? map - static_cast<int64_t>(gi) * UNITS : slot - static_cast<int64_t>(before) * UNITS;
        const int n = place < 2 ? gi : before, k0 = n * (place & 1) / 2, k1 = n * ((place & 1) + 1) / 2;
        Map2 run{splat2(1.f), splat2(0.f)};
        for (int k = k0; k < k1; k += 4) {
            ulonglong2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k + j < k1) v[j] = peek2(list + static_cast<int64_t>(k + j) * UNITS);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k + j < k1) {
                    const Map2 x = await2(list + static_cast<int64_t>(k + j) * UNITS, v[j], a);
                    run = k + j == k0 ? x : then<CUTS>(run, x);
                }
        }
        s.preA[place][lane] = run.A;
        s.preB[place][lane] = run.B;
        if (closes && gi + 1 < a.span) {   // the group's map waits for nothing but its chunks'
            __syncwarp();
            if (place != 1) asm volatile("bar.sync 1, 96;" ::: "memory");   // three of the warps
            if (place == 0) {
                const Map2 chunks = then<CUTS>(Map2{s.preA[2][lane], s.preB[2][lane]}, Map2{s.preA[3][lane], s.preB[3][lane]});
                publish2(map, then<CUTS>(chunks, all));
            }
        }
        if (place == 1) {
            if (sp > 0) h = await2(end - UNITS, peek2(end - UNITS), a).B;
            s.end[lane] = h;
        }
        __syncthreads();
        between();
        h = s.end[lane];
        if (gi + before > 0)
#pragma unroll
            for (int w = 0; w < NW; ++w) h = apply<CUTS>(Map2{s.preA[w][lane], s.preB[w][lane]}, h);
        if (!ok) h = nan;
        if (place == 0 && closes_span) publish2(end, Map2{splat2(0.f), apply<CUTS>(all, h)});
    }
    for (int w = 0; w < place; ++w) h = apply<CUTS>(warps_map(w), h);
    return h;
}

// A pack's segments at a warp's SEG steps from t0: lane r < SEG has the segment of step
// t0 + r, and whether the step is its first or its last (bit r of the masks).
template <int SEG>
__device__ __forceinline__ int segments_at(const RecArgs &a, int t0, int lane, uint32_t &heads, uint32_t &tails) {
    const int t = t0 + lane;
    int seg = 0;
    bool head = false, tail = false;
    if (lane < SEG && t < a.T) {
        seg = segment_of(a, t);
        head = __ldg(a.cu + seg) == t;
        tail = __ldg(a.cu + seg + 1) == t + 1;
    }
    heads = __ballot_sync(FULL_MASK, head);
    tails = __ballot_sync(FULL_MASK, tail);
    return seg;
}

// bounded wait for a tile's copies; after one that gave up the copies are seen through
__device__ __forceinline__ bool tile_is_there(uint64_t *bar, uint32_t parity, const RecArgs &a) {
    if (mbar_wait_bounded(bar, parity, a.wait_ns, a.error)) return true;
    mbar_wait_bounded(bar, parity, SETTLE_NS, a.error);
    return false;
}

// ---------------------------------------------------------------- forward
// tiles: FORWARD_TILES of them in shared memory
template <typename TS, bool WIDE, int MODE>
__device__ __forceinline__ void forward_tiles(const CUtensorMap *tmP, const CUtensorMap *tmH, const RecArgs &a, Shared &s, TS *tiles) {
    using Form = Shape<TS, WIDE>;
    constexpr int SEG = Form::SEG, PLANE = Form::PLANE, TERMS = 5;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto start = [&](uint32_t tile, int buf) {   // the copies of a tile
        const Place p = place_of<Form::L, false, MODE>(a, tile);
        mbar_arrive_expect_tx(&s.bar[buf], 3u * PLANE * sizeof(TS));
#pragma unroll
        for (int g = 0; g < 3; ++g)
            tma_load_3d(tiles + (buf * 3 + g) * PLANE, tmP, &s.bar[buf], g * a.d + p.u0, p.t0, p.b);
    };
    const uint32_t n_tiles = tiles_of<MODE>(a);
    if (tid == 0) {
        mbar_init(&s.bar[0], 1);
        mbar_init(&s.bar[1], 1);
        fence_mbar_init();
        s.tile[0] = atomicAdd(a.ticket, 1u);
        if (s.tile[0] < n_tiles) start(s.tile[0], 0);
    }
    __syncthreads();
    for (int it = 0;; ++it) {
        const int buf = WIDE ? it & 1 : 0;
        const uint32_t tile = s.tile[it & 1];
        if (tile >= n_tiles) break;
        const Place p = place_of<Form::L, false, MODE>(a, tile);
        const int u = p.u0 + 2 * lane, r0 = warp * SEG;
        const bool uok = u < a.d;
        const UnitWeights w = weights_of(a.params, a.d, u, uok);
        TS *const mine = tiles + buf * 3 * PLANE + r0 * UNITS + 2 * lane;
        uint32_t heads = 0, tails = 0;
        int seg = p.b;
        if (MODE == PACK) seg = segments_at<SEG>(a, p.t0 + r0, lane, heads, tails);
        else if (p.t_end - 1 - p.t0 - r0 >= 0 && p.t_end - 1 - p.t0 - r0 < SEG) tails = 1u << (p.t_end - 1 - p.t0 - r0);
        const bool starts = p.q < a.group * a.span && a.state != nullptr;   // in the first span
        if (MODE == PLAN && (starts || tails != 0)) seg = segment_of(a, p.t0);
        float2 first = splat2(0.f);   // what the first span starts from
        if (MODE != PACK && starts) first = two_of(a.state + static_cast<int64_t>(seg) * a.d + u, uok);
        // state before a segment's first step
        auto state_at = [&](int r) {
            const int sg = __shfl_sync(FULL_MASK, seg, r);
            return two_of(a.state + static_cast<int64_t>(sg) * a.d + u, uok && a.state != nullptr);
        };
        uint32_t next = 0;
        if (WIDE && tid == 0) next = atomicAdd(a.ticket, 1u);
        const bool ok = tile_is_there(&s.bar[buf], (WIDE ? it >> 1 : it) & 1, a);
        float2 da[SEG], du[SEG];
        Map2 m{splat2(1.f), splat2(0.f)};
        auto compose = [&](auto special) {
#pragma unroll
            for (int i = 0; i < SEG; ++i) {
                forward_gates<TERMS>(load2(mine + i * UNITS), load2(mine + PLANE + i * UNITS), load2(mine + 2 * PLANE + i * UNITS),
                                     w, da[i], du[i]);
                if (decltype(special)::value && (heads >> i & 1u)) {
                    m.B = fma2(da[i], state_at(i), du[i]);
                    m.A = splat2(-0.f);
                } else {
                    m.B = fma2(da[i], m.B, du[i]);
                    m.A = mul2(da[i], m.A);
                }
            }
        };
        if (MODE == PACK && heads != 0) compose(std::true_type{});
        else compose(std::false_type{});
        if (WIDE && tid == 0) s.tile[(it + 1) & 1] = next;
        if (WIDE && lane == 0) bulk_wait_read<0>();   // this warp's result has left the tile before
        float2 h = carry_into<WIDE, false, MODE == PACK>(a, s, it, p, warp, lane, m, first, ok, [&]() {
            if (tid == 0) {
                if (WIDE && next < n_tiles) start(next, buf ^ 1);
            }
        });
        auto write = [&](auto special) {
#pragma unroll
            for (int i = 0; i < SEG; ++i) {
                if (decltype(special)::value && MODE == PACK && (heads >> i & 1u)) h = state_at(i);
                h = fma2(da[i], h, du[i]);
                store2(mine + i * UNITS, h);
                if (decltype(special)::value && (tails >> i & 1u) && a.last != nullptr) {
                    const int sg = MODE == PACK ? __shfl_sync(FULL_MASK, seg, i) : seg;
                    if (uok) *reinterpret_cast<float2 *>(a.last + static_cast<int64_t>(sg) * a.d + u) = h;
                }
            }
        };
        if ((heads | tails) != 0) write(std::true_type{});
        else write(std::false_type{});
        fence_proxy_async_smem();
        __syncwarp();
        if (MODE == PLAN && p.t_end - p.t0 < Form::L) {   // the steps after the segment are the next one's
            for (int i = 0; i < SEG && p.t0 + r0 + i < p.t_end; ++i)
                if (uok) store2(static_cast<TS *>(a.H_out) + static_cast<int64_t>(p.t0 + r0 + i) * a.d + u, load2(mine + i * UNITS));
        } else if (lane == 0 && p.t0 + r0 < a.T) {
            tma_store_3d(tmH, mine, p.u0, p.t0 + r0, p.b);
            bulk_commit();
        }
        if (!WIDE) {   // (else s.tile was written before this tile's barrier, and the shared maps alternate)
            if (tid == 0) s.tile[(it + 1) & 1] = next = atomicAdd(a.ticket, 1u);
            if (lane == 0) bulk_wait_read<0>();
            __syncthreads();
            if (tid == 0 && next < n_tiles) start(next, 0);
        }
    }
    if (lane == 0) bulk_wait_read<0>();   // the tiles outlive the stores' reads
}

template <typename TS, bool WIDE, int MODE>
__global__ void __launch_bounds__(THREADS, (Shape<TS, WIDE>::FORWARD_CTAS))
    k_forward(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmH, const RecArgs a) {
    extern __shared__ __align__(128) unsigned char dsmem[];
    __shared__ Shared s;
    dependents_may_launch();
    wait_for_prerequisites();
    forward_tiles<TS, WIDE, MODE>(&tmP, &tmH, a, s, reinterpret_cast<TS *>(dsmem));
}

// a pack by its segments (a), or by the time axis (cut)
template <typename TS>
__global__ void __launch_bounds__(THREADS, (Shape<TS, true>::FORWARD_CTAS))
    k_forward_pack(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmH, const RecArgs a, const RecArgs cut) {
    extern __shared__ __align__(128) unsigned char dsmem[];
    __shared__ Shared s;
    dependents_may_launch();
    wait_for_prerequisites();
    if (by_segments(a.plan)) forward_tiles<TS, true, PLAN>(&tmP, &tmH, a, s, reinterpret_cast<TS *>(dsmem));
    else forward_tiles<TS, false, PACK>(&tmP, &tmH, cut, s, reinterpret_cast<TS *>(dsmem));
}

// ---------------------------------------------------------------- backward
// shared -> global store of a block of dL/dP through the 4-D map (d, block, T, B)
__device__ __forceinline__ void store_block(const CUtensorMap *map, const void *src, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// The tensor maps of a backward call, as the kernels take them
#define NRNN_BACKWARD_MAPS                                                                                    \
    const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmG, \
        const __grid_constant__ CUtensorMap tmGP
using Sums = float2[3][NW][32];

// Ps: one tile in shared memory: P, H, gH
template <typename TS, bool WIDE, int MODE>
__device__ __forceinline__ void backward_tiles(const CUtensorMap *tmP, const CUtensorMap *tmH, const CUtensorMap *tmG,
                                               const CUtensorMap *tmGP, const RecArgs &a, Shared &s, Sums &sums, TS *const Ps) {
    using Form = Shape<TS, WIDE>;
    constexpr int SEG = Form::SEG, PLANE = Form::PLANE, TERMS = sizeof(TS) == 2 ? 3 : 5;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    TS *const Hs = Ps + 3 * PLANE, *const Gs = Hs + PLANE;
    auto start = [&](uint32_t tile) {
        const Place p = place_of<Form::L, true, MODE>(a, tile);
        mbar_arrive_expect_tx(&s.bar[0], 5u * PLANE * sizeof(TS));
#pragma unroll
        for (int g = 0; g < 3; ++g) tma_load_3d(Ps + g * PLANE, tmP, &s.bar[0], g * a.d + p.u0, p.t0, p.b);
        tma_load_3d(Hs, tmH, &s.bar[0], p.u0, p.t0, p.b);
        tma_load_3d(Gs, tmG, &s.bar[0], p.u0, p.t0, p.b);
    };
    const uint32_t n_tiles = tiles_of<MODE>(a);
    if (tid == 0) {
        mbar_init(&s.bar[0], 1);
        fence_mbar_init();
        s.tile[0] = atomicAdd(a.ticket, 1u);
        if (s.tile[0] < n_tiles) start(s.tile[0]);
    }
    __syncthreads();
    for (int it = 0;; ++it) {
        const uint32_t tile = s.tile[it & 1];
        if (tile >= n_tiles) break;
        const Place p = place_of<Form::L, true, MODE>(a, tile);
        const int u = p.u0 + 2 * lane, r0 = warp * SEG;
        const bool uok = u < a.d;
        const UnitWeights w = weights_of(a.params, a.d, u, uok);
        TS *const mine = Ps + r0 * UNITS + 2 * lane;
        const TS *const h_mine = Hs + r0 * UNITS + 2 * lane, *const g_mine = Gs + r0 * UNITS + 2 * lane;
        uint32_t heads = 0, tails = 0;
        int seg = p.b;
        const int valid = MODE == PLAN ? p.t_end - p.t0 - r0 : SEG;   // steps of this warp before the segment's end
        if (MODE == PACK) {
            seg = segments_at<SEG>(a, p.t0 + r0, lane, heads, tails);
        } else {
            const int end = p.t_end - 1 - p.t0 - r0;
            if (end >= 0 && end < SEG) tails = 1u << end;
            if (MODE == PLAN ? p.q + 1 == p.nq && warp == 0 : p.t0 + r0 == 0) heads = 1u;
            if (MODE == PLAN && (heads | tails) != 0) seg = segment_of(a, p.t0);
        }
        auto row_of = [&](int r) { return static_cast<int64_t>(MODE == PACK ? __shfl_sync(FULL_MASK, seg, r) : seg) * a.d + u; };
        float2 before0 = splat2(0.f);   // H at the step before this warp's first
        if (warp == 0 && p.t0 > 0 && uok)
            before0 = load2(static_cast<const TS *>(a.H) + (static_cast<int64_t>(p.b) * a.T + p.t0 - 1) * a.d + u);
        const bool ok = tile_is_there(&s.bar[0], it & 1, a);
        if (warp > 0) before0 = load2(h_mine - UNITS);
        // nu_{t+1} -> nu_t = a_t (gH_t + nu_{t+1}), the last step first; a sequence's last
        // step starts from the gradient of its last state
        float2 dr[SEG], de[SEG];   // r, (1 - r) / r
        Map2 m{splat2(1.f), splat2(0.f)};
        auto compose = [&](auto special) {
#pragma unroll
            for (int i = SEG - 1; i >= 0; --i) {
                if (MODE == PLAN && decltype(special)::value && i >= valid) continue;   // the next segment's
                de[i] = falling(load2(mine + i * UNITS), w.nb_a);
                dr[i] = rcp_2(add2(de[i], splat2(1.f)));
                const float2 decay = decay_of<TERMS>(mul2(w.fall2, dr[i]));
                if (decltype(special)::value && (tails >> i & 1u)) {
                    m.B = two_of(a.g_last + row_of(i), uok && a.g_last != nullptr);
                    m.A = splat2(-0.f);
                }
                m.B = mul2(decay, add2(load2(g_mine + i * UNITS), m.B));
                m.A = mul2(decay, m.A);
            }
        };
        if (tails != 0 || valid < SEG) compose(std::true_type{});
        else compose(std::false_type{});
        uint32_t next = 0;
        float2 nu = carry_into<WIDE, true, MODE == PACK>(a, s, it, p, NW - 1 - warp, lane, m, splat2(0.f), ok, [&]() {
            if (WIDE && tid == 0) s.tile[(it + 1) & 1] = next = atomicAdd(a.ticket, 1u);
        });
        float2 g_wr = splat2(0.f), g_ba = splat2(0.f), g_bi = splat2(0.f);
        auto write = [&](auto special) {
#pragma unroll
            for (int i = SEG - 1; i >= 0; --i) {
                constexpr bool SPECIAL = decltype(special)::value;
                if (MODE == PLAN && SPECIAL && i >= valid) continue;
                if (SPECIAL && (tails >> i & 1u)) nu = two_of(a.g_last + row_of(i), uok && a.g_last != nullptr);
                const float2 ei = falling(load2(mine + PLANE + i * UNITS), w.nb_i), gi = rcp_2(add2(ei, splat2(1.f)));
                const float2 v = load2(mine + 2 * PLANE + i * UNITS);
                const float2 r = dr[i], z = mul2(w.fall2, r);
                float2 q;                                                 // a^2 - 1
                const float2 decay = decay_of<TERMS>(z, q);
                const float2 rs = make_float2(rsqrt_or_zero(-q.x), rsqrt_or_zero(-q.y));
                const float2 msq = mul2(q, rs), over = mul2(decay, rs);   // -s, a / s
                float2 before = i > 0 ? load2(h_mine + (i - 1) * UNITS) : before0;
                if (SPECIAL && (heads >> i & 1u)) before = two_of(a.state + row_of(i), uok && a.state != nullptr);
                const float2 G = add2(load2(g_mine + i * UNITS), nu);
                nu = mul2(decay, G);
                if (SPECIAL && (heads >> i & 1u) && a.g_state != nullptr) {
                    const int64_t at = row_of(i);
                    if (uok) *reinterpret_cast<float2 *>(a.g_state + at) = nu;
                }
                const float2 ngi = mul2(gi, splat2(-1.f)), miv = mul2(ngi, v);
                // w r with w = nu (before - over i v); then gP_a = -rate w r (1 - r), 1 - r = e r
                const float2 wr = mul2(mul2(nu, r), fma2(over, miv, before));
                const float2 ga = mul2(wr, mul2(mul2(z, splat2(0.6931471806f)), de[i]));   // -rate r = z ln 2
                const float2 mGs = mul2(G, msq);
                const float2 gv = mul2(mGs, ngi), gp = mul2(mul2(mGs, miv), mul2(ei, gi));
                g_wr = add2(g_wr, wr);
                g_ba = add2(g_ba, ga);
                g_bi = add2(g_bi, gp);
                store2(mine + i * UNITS, ga);
                store2(mine + PLANE + i * UNITS, gp);
                store2(mine + 2 * PLANE + i * UNITS, gv);
            }
        };
        if ((heads | tails) != 0 || valid < SEG) write(std::true_type{});
        else write(std::false_type{});
        if (!WIDE && tid == 0) s.tile[(it + 1) & 1] = next = atomicAdd(a.ticket, 1u);
        sums[0][warp][lane] = mul2(g_wr, splat2(-1.f));
        sums[1][warp][lane] = g_ba;
        sums[2][warp][lane] = g_bi;
        fence_proxy_async_smem();
        __syncwarp();
        if (MODE == PLAN && p.t_end - p.t0 < Form::L) {
            for (int i = 0; i < SEG && i < valid; ++i)
#pragma unroll
                for (int g = 0; g < 3; ++g)
                    if (uok)
                        store2(static_cast<TS *>(a.gP) + (static_cast<int64_t>(p.t0 + r0 + i) * 3 + g) * a.d + u,
                               load2(mine + g * PLANE + i * UNITS));
        } else if (lane == 0 && p.t0 + r0 < a.T) {
#pragma unroll
            for (int g = 0; g < 3; ++g) store_block(tmGP, Ps + g * PLANE + r0 * UNITS, p.u0, g, p.t0 + r0, p.b);
            bulk_commit();
            bulk_wait_read<0>();
        }
        __syncthreads();
        if (tid == 0 && next < n_tiles) start(next);
        if (warp < 3) {
            float2 t = sums[warp][0][lane];
#pragma unroll
            for (int k = 1; k < NW; ++k) t = add2(t, sums[warp][k][lane]);
            float *to = a.part + (p.at * 3 + warp) * UNITS + 2 * lane;
            *reinterpret_cast<float2 *>(to) = t;
        }
        // (the next tile's first barrier lies between these reads and its sums)
    }
}

template <typename TS, bool WIDE, int MODE>
__global__ void __launch_bounds__(THREADS, (Shape<TS, WIDE>::BACKWARD_CTAS)) k_backward(NRNN_BACKWARD_MAPS, const RecArgs a) {
    extern __shared__ __align__(128) unsigned char dsmem[];
    __shared__ Shared s;
    __shared__ Sums sums;
    dependents_may_launch();
    wait_for_prerequisites();
    backward_tiles<TS, WIDE, MODE>(&tmP, &tmH, &tmG, &tmGP, a, s, sums, reinterpret_cast<TS *>(dsmem));
}

template <typename TS>
__global__ void __launch_bounds__(THREADS, (Shape<TS, true>::BACKWARD_CTAS))
    k_backward_pack(NRNN_BACKWARD_MAPS, const RecArgs a, const RecArgs cut) {
    extern __shared__ __align__(128) unsigned char dsmem[];
    __shared__ Shared s;
    __shared__ Sums sums;
    dependents_may_launch();
    wait_for_prerequisites();
    if (by_segments(a.plan)) backward_tiles<TS, true, PLAN>(&tmP, &tmH, &tmG, &tmGP, a, s, sums, reinterpret_cast<TS *>(dsmem));
    else backward_tiles<TS, false, PACK>(&tmP, &tmH, &tmG, &tmGP, cut, s, sums, reinterpret_cast<TS *>(dsmem));
}

// Sums of the parameters' gradients over rows and chunks, in order: a CTA takes a unit
// tile and one of JOIN_SLICES shares of (row, chunk); the CTA that ends last, by a
// counter, adds the shares.
constexpr int JOIN_SLICES = 32, JOIN_THREADS = 3 * UNITS;

__global__ void __launch_bounds__(JOIN_THREADS)
    k_join(const float *part, int rows, int n_ut, int n_chunks, const int4 *plan, int cut_chunks, int d, float *share,
           uint32_t *count, float *gparams) {
    __shared__ bool is_last;
    dependents_may_launch();
    wait_for_prerequisites();
    const int ut = blockIdx.x, slice = blockIdx.y, j = threadIdx.x;
    if (plan != nullptr && !by_segments(plan)) {
        plan = nullptr;
        n_chunks = cut_chunks;
    }
    // (tiles are counted in 32 bits; a plan: one row)
    const uint32_t all = plan != nullptr ? static_cast<uint32_t>(plan[0].x) : static_cast<uint32_t>(rows) * n_chunks;
    const uint32_t k0 = static_cast<uint64_t>(all) * slice / JOIN_SLICES, k1 = static_cast<uint64_t>(all) * (slice + 1) / JOIN_SLICES;
    auto at = [&](uint32_t k) {
        const uint32_t b = k / static_cast<uint32_t>(n_chunks), q = k - b * n_chunks;
        return part[((static_cast<int64_t>(b) * n_ut + ut) * n_chunks + q) * JOIN_THREADS + j];
    };
    float t[8] = {};
    uint32_t k = k0;
    for (; k + 8 <= k1; k += 8)
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] += at(k + e);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (k + e < k1) t[e] += at(k + e);
#pragma unroll
    for (int e = 4; e > 0; e /= 2)
        for (int i = 0; i < e; ++i) t[i] += t[i + e];
    share[(static_cast<int64_t>(ut) * JOIN_SLICES + slice) * JOIN_THREADS + j] = t[0];
    __threadfence();
    __syncthreads();
    if (j == 0) is_last = atomicAdd(count + ut, 1u) == JOIN_SLICES - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    float sum = 0.f;
#pragma unroll 8
    for (int e = 0; e < JOIN_SLICES; ++e)
        sum += __ldcg(share + (static_cast<int64_t>(ut) * JOIN_SLICES + e) * JOIN_THREADS + j);
    const int u = ut * UNITS + j % UNITS;
    if (u < d) gparams[static_cast<int64_t>(j / UNITS) * d + u] = sum;
}

// A pack goes by its segments where the longest of them has at most 1 / LONGEST of all tiles:
// its chain takes a chunk in 0.45 to 0.7 us however few others are left, about as long as the
// machine takes for that many tiles.  262144 x 512 in 64 segments of which one has 16384,
// 32768 or 250000 steps, by segments and by the time axis: forward fp32 475, 665, 3795 and 575
// us, bf16 262, 354, 1818 and 352; backward 854, 1126, 4890 and 838, 568, 727, 3112 and 585.
template <bool REVERSE> constexpr int64_t LONGEST = REVERSE ? 140 : 100;

// Clears a call's counters, error word and slots.  Sequences without a step hand their state (or its
// gradient) on; with no steps at all the parameters' gradients are zeros.  With a plan the
// first CTA builds it, if the call is to go by it, and clears nothing.
constexpr int PREPARE_THREADS = 256;

template <int L>
__global__ void __launch_bounds__(PREPARE_THREADS)
    k_prepare(uint4 *clear, int64_t n16, const int32_t *cu, int rows, int T, int d, const float *in, float *out, float *zeros,
              int4 *plan, bool reverse) {
    extern __shared__ int plan_space[];
    dependents_may_launch();
    wait_for_prerequisites();
    int first = 0;
    if (plan != nullptr) {
        if (blockIdx.x == 0) {
            __shared__ int longest, all;
            if (threadIdx.x == 0) longest = all = 0;
            __syncthreads();
            int most = 0, sum = 0;
            for (int i = threadIdx.x; i < rows; i += PREPARE_THREADS) {
                const int c = (max(0, __ldg(cu + i + 1) - __ldg(cu + i)) + L - 1) / L;
                most = max(most, c);
                sum += c;
            }
            atomicMax(&longest, most);
            atomicAdd(&all, sum);
            __syncthreads();
            const int64_t tiles = static_cast<int64_t>(all) * ((d + UNITS - 1) / UNITS);
            const bool segments = longest * (reverse ? LONGEST<true> : LONGEST<false>) <= tiles;
            if (segments) build_pack_plan<PREPARE_THREADS, L>(cu, rows, (T + L - 1) / L, reverse, plan, plan_space);
            if (threadIdx.x == 0) plan[0] = make_int4(all, segments, 0, 0);
            return;
        }
        first = 1;
    }
    const int64_t i0 = static_cast<int64_t>(blockIdx.x - first) * PREPARE_THREADS + threadIdx.x,
                  step = static_cast<int64_t>(gridDim.x - first) * PREPARE_THREADS;
    for (int64_t i = i0; i < n16; i += step) clear[i] = make_uint4(0u, 0u, 0u, 0u);
    if (out != nullptr && (cu != nullptr || T == 0))
        for (int64_t i = i0; i < static_cast<int64_t>(rows) * d; i += step) {
            const int64_t row = i / d;
            if (cu == nullptr || __ldg(cu + row) >= __ldg(cu + row + 1)) out[i] = in != nullptr ? in[i] : 0.f;
        }
    if (zeros != nullptr)
        for (int64_t i = i0; i < 3 * static_cast<int64_t>(d); i += step) zeros[i] = 0.f;
}

// ---------------------------------------------------------------- one step
template <typename TS>
__global__ void __launch_bounds__(256)
    k_step(const TS *P, const float *params, const float *state, int64_t pairs, int d, TS *h_out, float *last) {
    dependents_may_launch();
    wait_for_prerequisites();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= pairs) return;
    const int64_t slot = i / (d / 2);
    const int u = 2 * static_cast<int>(i - slot * (d / 2));
    const TS *p = P + slot * 3 * d + u;
    const float2 pa = load2(p), pi = load2(p + d), v = load2(p + 2 * d);
    const float2 before = two_of(state + slot * d + u, state != nullptr);
    float2 a, x;
    forward_gates<5>(pa, pi, v, weights_of(params, d, u, true), a, x);
    const float2 h = fma2(a, before, x);
    store2(h_out + slot * d + u, h);
    *reinterpret_cast<float2 *>(last + slot * d + u) = h;
}

// ---------------------------------------------------------------- host side
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

struct Layout {
    bool wide;
    int64_t n_ut, n_cols, n_chunks, group, span, n_tiles;
    int64_t cut_chunks;   // with a plan: chunks of the time axis
    int64_t slots, maps, ends, cleared, plan, part, share, total;   // plan 0: none
};
// the look-back where the warps share the maps before: a hop takes 2 to 3 us, and a chunk
// reads half a group's and half a span's maps on average
constexpr int64_t GROUP = 16, SPAN = 16;

// Columns from which a call takes the WIDE form.  bf16 of 64 and 128 columns (16384 and 8192
// steps) forward 188 and 128 us, 138 and 133 the other, backward 267 and 220, 240 and 243;
// fp32 of 64, 128, 256 columns forward 2.7, 4.1, 6.2 TB/s, the other 5.0, backward of 128
// 6.1, of 64 the other 4.9.
constexpr int64_t wide_columns(int dtype, bool backward) { return dtype == NRNN_F32 && !backward ? 256 : 128; }

// num_segments > 0: a pack.  Its segments are columns where they are enough of them for
// the WIDE form, long enough (a segment adds a short chunk), and the plan is small; there is
// room for both ways, which share the slots and sums.
Layout layout_of(int64_t B, int64_t T, int64_t d, int dtype, int64_t num_segments, bool backward) {
    Layout y{};
    const int64_t wide_steps = dtype == NRNN_BF16 ? Shape<__nv_bfloat16, true>::L : Shape<float, true>::L;
    const int64_t steps = dtype == NRNN_BF16 ? Shape<__nv_bfloat16, false>::L : Shape<float, false>::L;
    y.n_ut = ceil_div(d, UNITS);
    const bool plan = B == 1 && num_segments >= 2 && num_segments <= PACK_PLAN_MAX_S && ceil_div(T, wide_steps) <= PACK_PLAN_MAX_CHUNKS &&
                      8 * num_segments <= ceil_div(T, wide_steps) && num_segments * y.n_ut >= wide_columns(dtype, backward);
    y.n_cols = B * y.n_ut;
    y.wide = plan || y.n_cols >= wide_columns(dtype, backward);
    y.n_chunks = ceil_div(T, y.wide ? wide_steps : steps) + (plan ? num_segments : 0);
    y.cut_chunks = plan ? ceil_div(T, steps) : 0;
    y.group = !y.wide ? GROUP : backward ? WIDE_GROUP<true> : WIDE_GROUP<false>;
    y.span = y.wide ? 1 : SPAN;
    const int64_t groups = ceil_div(plan ? y.cut_chunks : y.n_chunks, GROUP);
    y.n_tiles = y.n_cols * y.n_chunks;
    int64_t at = 256 + up256(4 * y.n_ut);   // ticket, error; the join's counters
    auto take = [&](int64_t per_column) {
        const int64_t o = at;
        at += 8 * UNITS * y.n_cols * per_column;
        return o;
    };
    y.slots = take(y.n_chunks);
    y.maps = take(y.wide && !plan ? 0 : groups);
    y.ends = take(y.wide && !plan ? 0 : ceil_div(groups, SPAN));
    y.cleared = at;
    if (plan) {
        y.plan = at;
        at += up256(16 * (1 + y.n_chunks));
    }
    y.part = at;
    if (backward) {
        at += up256(4 * 3 * UNITS * y.n_tiles);
        y.share = at;
        at += up256(4 * 3 * UNITS * JOIN_SLICES * y.n_ut);
    }
    y.total = at;
    return y;
}

int check(const void *P, int dtype, const float *params, int64_t B, int64_t T, int64_t d,
          const int32_t *cu, int64_t S) {
    if (dtype != NRNN_F32 && dtype != NRNN_BF16) return NRNN_ERR_INVALID_ARG;
    if (B < 0 || T < 0 || d <= 0 || S < 0) return NRNN_ERR_INVALID_ARG;
    if (B > INT32_MAX || T > INT32_MAX || d > (1 << 24) || S > INT32_MAX - 1 || d % 8 != 0)
        return NRNN_ERR_UNSUPPORTED;
    // tiles are counted in 32 bits
    if (B > 0 && T > 0 && ceil_div(T, 32) > INT32_MAX / (B * ceil_div(d, UNITS))) return NRNN_ERR_UNSUPPORTED;
    if (cu != nullptr && (B != 1 || S < 1)) return NRNN_ERR_CU_SEQLENS;
    if (params == nullptr || !aligned16(params)) return NRNN_ERR_INVALID_ARG;
    if (B * T > 0 && (P == nullptr || !aligned16(P))) return NRNN_ERR_INVALID_ARG;
    return NRNN_OK;
}

bool usable(const void *ws, size_t have, int64_t need) {
    return ws != nullptr && reinterpret_cast<uintptr_t>(ws) % 256 == 0 && have >= static_cast<size_t>(need);
}

RecArgs args_of(const Layout &y, const float *params, const float *state, const int32_t *cu, int64_t rows, int64_t T,
                int64_t d, unsigned char *ws) {
    RecArgs a{};
    a.params = params; a.state = state; a.cu = cu;
    a.rows = static_cast<int>(rows); a.T = static_cast<int>(T); a.d = static_cast<int>(d);
    a.n_ut = static_cast<int>(y.n_ut); a.n_cols = static_cast<int>(y.n_cols); a.n_chunks = static_cast<int>(y.n_chunks);
    a.group = static_cast<int>(y.group);
    a.span = static_cast<int>(y.span);
    a.n_tiles = static_cast<uint32_t>(y.n_tiles);
    a.ticket = reinterpret_cast<uint32_t *>(ws);
    a.error = a.ticket + 1;
    a.slots = reinterpret_cast<unsigned long long *>(ws + y.slots);
    a.maps = reinterpret_cast<unsigned long long *>(ws + y.maps);
    a.ends = reinterpret_cast<unsigned long long *>(ws + y.ends);
    a.plan = y.plan != 0 ? reinterpret_cast<const int4 *>(ws + y.plan) : nullptr;
    a.part = reinterpret_cast<float *>(ws + y.part);
    a.wait_ns = wait_limit_ns();
    return a;
}

// the arguments of a call with a plan that goes by the time axis
RecArgs cut_args(const Layout &y, RecArgs a) {
    a.n_chunks = static_cast<int>(y.cut_chunks);
    a.group = static_cast<int>(GROUP);
    a.span = static_cast<int>(SPAN);
    a.n_tiles = static_cast<uint32_t>(y.n_cols * y.cut_chunks);
    a.plan = nullptr;
    return a;
}

template <int L>
cudaError_t prepare(const Layout &y, const RecArgs &a, unsigned char *ws, const float *in, float *out, float *zeros,
                    bool reverse, cudaStream_t s) {
    const int64_t n16 = (y.n_tiles > 0 ? y.cleared : 256) / 16;   // (without steps: the error word's)
    const int64_t most = n16 > static_cast<int64_t>(a.rows) * a.d ? n16 : static_cast<int64_t>(a.rows) * a.d;
    int64_t b = ceil_div(most, PREPARE_THREADS);
    b = b < 1 ? 1 : b < 1216 ? b : 1216;
    size_t smem = 0;
    int4 *plan = nullptr;
    if (y.plan != 0) {
        static std::atomic<unsigned long long> configured{0};
        cudaError_t e = once_per_device(configured, [](int) {
            return cudaFuncSetAttribute(k_prepare<L>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(pack_plan_smem(PACK_PLAN_MAX_S, PACK_PLAN_MAX_CHUNKS)));
        });
        if (e != cudaSuccess) return e;
        plan = reinterpret_cast<int4 *>(ws + y.plan);
        smem = pack_plan_smem(a.rows, static_cast<int>(ceil_div(a.T, L)));
        b += 1;   // the first one plans
    }
    return launch_dependent(k_prepare<L>, static_cast<unsigned>(b), PREPARE_THREADS, smem, s, reinterpret_cast<uint4 *>(ws), n16,
                            a.cu, a.rows, a.T, a.d, in, out, zeros, plan, reverse);
}
cudaError_t prepare(int dtype, const Layout &y, const RecArgs &a, unsigned char *ws, const float *in, float *out, float *zeros,
                    bool reverse, cudaStream_t s) {
    return dtype == NRNN_BF16 ? prepare<Shape<__nv_bfloat16, true>::L>(y, a, ws, in, out, zeros, reverse, s)
                              : prepare<Shape<float, true>::L>(y, a, ws, in, out, zeros, reverse, s);
}

unsigned ctas_for(int64_t tiles, int per_sm) {
    const int64_t most = 152ll * per_sm;
    return static_cast<unsigned>(tiles < most ? tiles : most);
}

template <typename TS, bool WIDE, int MODE>
cudaError_t launch_forward(const Layout &y, const RecArgs &a, int dtype, const void *P, void *H, int64_t B, cudaStream_t s) {
    using Form = Shape<TS, WIDE>;
    static std::atomic<unsigned long long> configured{0};
    constexpr size_t smem = static_cast<size_t>(Form::FORWARD_TILES) * 3 * Form::PLANE * sizeof(TS);
    cudaError_t e = once_per_device(configured, [](int) {
        if constexpr (MODE == PLAN)
            return cudaFuncSetAttribute(k_forward_pack<TS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        else
            return cudaFuncSetAttribute(k_forward<TS, WIDE, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    });
    if (e != cudaSuccess) return e;
    CUtensorMap tmP, tmH;
    if (!make_map_steps(&tmP, P, dtype, 3 * a.d, a.T, B, UNITS, Form::L) ||
        !make_map_steps(&tmH, H, dtype, a.d, a.T, B, UNITS, Form::SEG))
        return cudaErrorUnknown;
    const unsigned ctas = ctas_for(y.n_tiles, Form::FORWARD_CTAS);
    if constexpr (MODE == PLAN) return launch_dependent(k_forward_pack<TS>, ctas, THREADS, smem, s, tmP, tmH, a, cut_args(y, a));
    else return launch_dependent(k_forward<TS, WIDE, MODE>, ctas, THREADS, smem, s, tmP, tmH, a);
}

template <typename TS, bool WIDE, int MODE>
cudaError_t launch_backward(const Layout &y, const RecArgs &a, int dtype, const void *P, const void *H, const void *gH,
                            void *gP, int64_t B, cudaStream_t s) {
    using Form = Shape<TS, WIDE>;
    static std::atomic<unsigned long long> configured{0};
    constexpr size_t smem = 5ull * Form::PLANE * sizeof(TS);
    cudaError_t e = once_per_device(configured, [](int) {
        if constexpr (MODE == PLAN)
            return cudaFuncSetAttribute(k_backward_pack<TS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        else
            return cudaFuncSetAttribute(k_backward<TS, WIDE, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    });
    if (e != cudaSuccess) return e;
    CUtensorMap tmP, tmH, tmG, tmGP;
    if (!make_map_steps(&tmP, P, dtype, 3 * a.d, a.T, B, UNITS, Form::L) ||
        !make_map_steps(&tmH, H, dtype, a.d, a.T, B, UNITS, Form::L) ||
        !make_map_steps(&tmG, gH, dtype, a.d, a.T, B, UNITS, Form::L) ||
        !make_map_gate_steps(&tmGP, gP, dtype, a.d, a.T, B, UNITS, Form::SEG))
        return cudaErrorUnknown;
    const unsigned ctas = ctas_for(y.n_tiles, Form::BACKWARD_CTAS);
    if constexpr (MODE == PLAN)
        return launch_dependent(k_backward_pack<TS>, ctas, THREADS, smem, s, tmP, tmH, tmG, tmGP, a, cut_args(y, a));
    else
        return launch_dependent(k_backward<TS, WIDE, MODE>, ctas, THREADS, smem, s, tmP, tmH, tmG, tmGP, a);
}

// launch<TS, WIDE, MODE>(args...) for the call
#define BY_MODE(launch, TS, y, pack, ...)                                                                         \
    ((y).plan != 0 ? launch<TS, true, PLAN>(y, __VA_ARGS__)                                                       \
     : (y).wide    ? ((pack) ? launch<TS, true, PACK>(y, __VA_ARGS__) : launch<TS, true, ROWS>(y, __VA_ARGS__))   \
                   : ((pack) ? launch<TS, false, PACK>(y, __VA_ARGS__) : launch<TS, false, ROWS>(y, __VA_ARGS__)))
#define BY_FORM(launch, y, dtype, pack, ...)                                        \
    ((dtype) == NRNN_BF16 ? BY_MODE(launch, __nv_bfloat16, y, pack, __VA_ARGS__)    \
                          : BY_MODE(launch, float, y, pack, __VA_ARGS__))

}  // namespace
}  // namespace nrnn

using namespace nrnn;

extern "C" {

size_t nrnn_linear_recurrence_workspace_bytes(int64_t B, int64_t T, int64_t d_h, int dtype,
                                              int64_t num_segments, int backward) {
    if (num_segments < 0 || (dtype != NRNN_F32 && dtype != NRNN_BF16) || B < 0 || T < 0 || d_h <= 0 || B > INT32_MAX ||
        T > INT32_MAX || d_h > (1 << 24) || (B > 0 && T > 0 && ceil_div(T, 32) > INT32_MAX / (B * ceil_div(d_h, UNITS))))
        return 0;
    return static_cast<size_t>(layout_of(B, T, d_h, dtype, num_segments, backward != 0).total);
}

int nrnn_linear_recurrence_forward(const void *preact, int dtype, const float *params, int64_t B,
                                   int64_t T, int64_t d_h, const int32_t *cu_seqlens,
                                   int64_t num_segments, const float *state, void *H, float *last,
                                   void *workspace, size_t ws_bytes, void *stream) {
    const int st = check(preact, dtype, params, B, T, d_h, cu_seqlens, num_segments);
    if (st != NRNN_OK) return st;
    const int64_t es = dtype == NRNN_BF16 ? 2 : 4, n = B * T * d_h;
    const int64_t rows = cu_seqlens != nullptr ? num_segments : B, sb = rows * d_h * 4;
    if ((n > 0 && (H == nullptr || !aligned16(H))) || !aligned16(state) || !aligned16(last) ||
        !outputs_apart({{H, n * es}, {last, sb}},
                       {{preact, 3 * n * es}, {params, 12 * d_h}, {state, sb}, {cu_seqlens, 4 * (rows + 1)}}))
        return NRNN_ERR_INVALID_ARG;
    const Layout y = layout_of(B, T, d_h, dtype, cu_seqlens != nullptr ? num_segments : 0, false);
    if (!usable(workspace, ws_bytes, y.total)) return NRNN_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    RecArgs a = args_of(y, params, state, cu_seqlens, rows, T, d_h, ws);
    a.last = last;
    a.H_out = H;
    cudaError_t e = prepare(dtype, y, a, ws, state, last, nullptr, false, s);
    if (e == cudaSuccess && n > 0) e = BY_FORM(launch_forward, y, dtype, cu_seqlens != nullptr, a, dtype, preact, H, B, s);
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

int nrnn_linear_recurrence_backward(const void *preact, int dtype, const float *params, int64_t B,
                                    int64_t T, int64_t d_h, const int32_t *cu_seqlens,
                                    int64_t num_segments, const float *state, const void *H,
                                    const void *gH, const float *g_last, void *gP, float *gparams,
                                    float *g_state, void *workspace, size_t ws_bytes, void *stream) {
    const int st = check(preact, dtype, params, B, T, d_h, cu_seqlens, num_segments);
    if (st != NRNN_OK) return st;
    const int64_t es = dtype == NRNN_BF16 ? 2 : 4, n = B * T * d_h;
    const int64_t rows = cu_seqlens != nullptr ? num_segments : B, sb = rows * d_h * 4;
    if (gparams == nullptr || !aligned16(gparams) || !aligned16(state) || !aligned16(g_last) || !aligned16(g_state) ||
        (n > 0 && (H == nullptr || gH == nullptr || gP == nullptr || !aligned16(H) || !aligned16(gH) || !aligned16(gP))) ||
        !outputs_apart({{gP, 3 * n * es}, {gparams, 12 * d_h}, {g_state, sb}},
                       {{preact, 3 * n * es}, {params, 12 * d_h}, {state, sb}, {cu_seqlens, 4 * (rows + 1)},
                        {H, n * es}, {gH, n * es}, {g_last, sb}}))
        return NRNN_ERR_INVALID_ARG;
    const Layout y = layout_of(B, T, d_h, dtype, cu_seqlens != nullptr ? num_segments : 0, true);
    if (!usable(workspace, ws_bytes, y.total)) return NRNN_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    RecArgs a = args_of(y, params, state, cu_seqlens, rows, T, d_h, ws);
    a.H = H;
    a.gP = gP;
    a.g_last = g_last;
    a.g_state = g_state;
    cudaError_t e = prepare(dtype, y, a, ws, g_last, g_state, n > 0 ? nullptr : gparams, true, s);
    if (e == cudaSuccess && n > 0) {
        e = BY_FORM(launch_backward, y, dtype, cu_seqlens != nullptr, a, dtype, preact, H, gH, gP, B, s);
        if (e == cudaSuccess) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(y.n_ut), JOIN_SLICES);
            cfg.blockDim = dim3(JOIN_THREADS);
            cfg.stream = s;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaLaunchKernelEx(&cfg, k_join, static_cast<const float *>(a.part), static_cast<int>(B), a.n_ut, a.n_chunks,
                                   a.plan, static_cast<int>(y.cut_chunks), a.d, reinterpret_cast<float *>(ws + y.share), reinterpret_cast<uint32_t *>(ws + 256), gparams);
        }
    }
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

int nrnn_linear_recurrence_step(const void *preact, int dtype, const float *params, int64_t slots,
                                int64_t d_h, const float *state, void *h, float *state_out,
                                void *stream) {
    const int st = check(preact, dtype, params, slots, 1, d_h, nullptr, 0);
    if (st != NRNN_OK) return st;
    const int64_t es = dtype == NRNN_BF16 ? 2 : 4, n = slots * d_h;
    if (n == 0) return NRNN_OK;
    if (h == nullptr || state_out == nullptr || !aligned16(h) || !aligned16(state_out) || !aligned16(state) ||
        !outputs_apart({{h, n * es}, {state_out, 4 * n}}, {{preact, 3 * n * es}, {params, 12 * d_h}}) ||
        !outputs_apart({{h, n * es}, {state != state_out ? state_out : nullptr, 4 * n}}, {{state, 4 * n}}))
        return NRNN_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t pairs = n / 2, blocks = ceil_div(pairs, 256);
    if (blocks > INT32_MAX) return NRNN_ERR_UNSUPPORTED;
    const cudaError_t e =
        dtype == NRNN_BF16
            ? launch_dependent(k_step<__nv_bfloat16>, static_cast<unsigned>(blocks), 256, 0, s,
                               static_cast<const __nv_bfloat16 *>(preact), params, state, pairs, static_cast<int>(d_h),
                               static_cast<__nv_bfloat16 *>(h), state_out)
            : launch_dependent(k_step<float>, static_cast<unsigned>(blocks), 256, 0, s, static_cast<const float *>(preact), params,
                               state, pairs, static_cast<int>(d_h), static_cast<float *>(h), state_out);
    return e == cudaSuccess ? NRNN_OK : NRNN_ERR_CUDA;
}

}  // extern "C"
