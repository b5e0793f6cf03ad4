// What the kernels of CTA pairs (tcgen05, cta_group::2) share: waits that one role's
// giving up ends for all, and fp32 values as bf16 planes.
#pragma once

#include "rows.cuh"
#include "tcgen05.cuh"

namespace nrnn {

constexpr uint64_t SETTLE_NS = 2000000000ull;   // for what is in flight after a wait gave up

// A: a kernel's arguments, with the call's error word (error) and the limit of a
// wait (wait_ns).

// mbar_wait_bounded that also ends when another role of the pair gave up, and tells
// both CTAs when it does
template <typename A>
__device__ __forceinline__ bool wait_or_abort(const A &a, uint64_t *bar, uint32_t parity,
                                              volatile uint32_t *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t hint = static_cast<uint32_t>(a.wait_ns < 1000000u ? a.wait_ns : 1000000u);
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (*abort != 0) return false;
        if (mbar_try_wait_hint(bar, parity, hint)) return true;
        if (globaltimer_ns() - t0 > a.wait_ns) {
            for (uint32_t r = 0; r < 2; ++r)
                cluster_store(cluster_addr(const_cast<const uint32_t *>(abort), r), 1u);
            atomicOr(a.error, 2u);
            return false;
        }
    }
}

// After a wait gave up, and both CTAs' roles have ended: sees through what is in flight.
// issued: stages that each CTA's producer started the copies of.  One that is ahead of
// the other (by at most the ring, whose stages are handed back to both at once) has
// copies that the stage's barrier, rank 0's, cannot complete on: it is brought to wait
// for that CTA's bytes alone.  By the issuing thread of rank 0.
template <int STAGES, typename A>
__device__ __forceinline__ void settle(const A &a, const volatile int *issued, uint64_t *full_bar,
                                       uint64_t *drain_bar, uint32_t bytes_1) {
    mma_commit_pair(drain_bar);
    mbar_wait_bounded(drain_bar, 0, SETTLE_NS, a.error);
    const int n0 = issued[0], n1 = issued[1], both = n0 < n1 ? n0 : n1, most = n0 < n1 ? n1 : n0;
    for (int i = both > STAGES ? both - STAGES : 0; i < most; ++i) {
        uint64_t *bar = &full_bar[i % STAGES];
        if (i >= both && n0 > n1) mbar_complete_tx(bar, bytes_1);              // was to come from rank 1
        else if (i >= both) mbar_arrive_expect_tx(bar, bytes_1);               // rank 0 never got there
        mbar_wait_bounded(bar, (i / STAGES) & 1, SETTLE_NS, a.error);
    }
}

// Two values as bf16, the nearest; or the type's largest where that is an infinity,
// so that a finite value less its first plane is a number.  (An infinity less the
// largest stays one, and its third plane is NaN.)
__device__ __forceinline__ __nv_bfloat162 finite_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return *reinterpret_cast<__nv_bfloat162 *>(&r);
}

// The first plane of v: the nearest bf16, or the one below in magnitude where that is
// an infinity but v (the lowest value, as a mask) is not, so that v less it is a number.
__device__ __forceinline__ float plane_of(float v) {
    const float h = __bfloat162float(__float2bfloat16_rn(v));
    return isinf(h) ? __bfloat162float(__float2bfloat16_rz(v)) : h;
}

// One row of `pitch` values (a multiple of 8) as bf16 planes, by the lanes of a warp;
// src null: zeros.  16 bytes out at a time; wide: 16 bytes in as well.
template <typename T>
__device__ __forceinline__ void copy_row(const T *src, __nv_bfloat16 *dst, int64_t plane, int d,
                                         int pitch, int lane, bool wide) {
#pragma unroll 4
    for (int c = lane * 8; c < pitch; c += 256) {
        float v[8];
        if (src != nullptr && wide) {
#pragma unroll
            for (int q = 0; q < 8; q += 16 / sizeof(T)) {
                float x[16 / sizeof(T)];
                load_f32<T, 16 / sizeof(T)>(src + c + q, x);
#pragma unroll
                for (int e = 0; e < static_cast<int>(16 / sizeof(T)); ++e) v[q + e] = x[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = src != nullptr && c + e < d ? to_f32(src[c + e]) : 0.f;
        }
#pragma unroll
        for (int p = 0; p < (sizeof(T) == 4 ? 3 : 1); ++p) {
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = sizeof(T) == 4 ? plane_of(v[e]) : v[e];
                v[e] -= h[e];
            }
            store_f32<__nv_bfloat16, 8>(dst + p * plane + c, h);
        }
    }
}
// rows of src can be read 16 bytes at a time
template <typename T> __device__ __forceinline__ bool wide_rows(const void *src, int d) {
    return d % 8 == 0 && (reinterpret_cast<uintptr_t>(src) & 15) == 0;
}

}  // namespace nrnn
