// Rows of (n, d) arrays as vectors: shared by the kernels that stream rows.
#pragma once

#include <initializer_list>

#include "nrnn_device.cuh"

namespace nrnn {

// programmatic dependent launch: the next kernel of the call may be scheduled now;
// wait until the one before has completed
__device__ __forceinline__ void dependents_may_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_prerequisites() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// VEC consecutive elements of a row as one load or store
template <typename T, int VEC> struct __align__(sizeof(T) * VEC) Pack { T v[VEC]; };

template <typename T, int VEC>
__device__ __forceinline__ void load_f32(const T *p, float (&f)[VEC]) {
    const Pack<T, VEC> r = *reinterpret_cast<const Pack<T, VEC> *>(p);
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = to_f32(r.v[e]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_f32(T *p, const float (&f)[VEC]) {
    Pack<T, VEC> r;
#pragma unroll
    for (int e = 0; e < VEC; ++e) r.v[e] = from_f32<T>(f[e]);
    *reinterpret_cast<Pack<T, VEC> *>(p) = r;
}

// elements per access: as wide as the row's alignment allows (at most 16
// bytes), but no wider than lets `lanes` lanes cover a narrow row
inline int vec_of(int elem, int64_t d, int lanes, std::initializer_list<const void *> ptrs) {
    int v = 16 / elem;
    while (v > 1) {
        bool ok = d % v == 0 && d > lanes * (v / 2);
        for (const void *p : ptrs) ok = ok && reinterpret_cast<uintptr_t>(p) % (v * elem) == 0;
        if (ok) break;
        v /= 2;
    }
    return v;
}

// calls f<T, VEC>(args...) for the storage type and access width
#define NRNN_BY_WIDTH(dtype, vec, f, ...)                                             \
    ((dtype) == NRNN_BF16                                                             \
         ? ((vec) == 8   ? f<__nv_bfloat16, 8>(__VA_ARGS__)                           \
            : (vec) == 4 ? f<__nv_bfloat16, 4>(__VA_ARGS__)                           \
            : (vec) == 2 ? f<__nv_bfloat16, 2>(__VA_ARGS__)                           \
                         : f<__nv_bfloat16, 1>(__VA_ARGS__))                          \
         : ((vec) == 4   ? f<float, 4>(__VA_ARGS__)                                   \
            : (vec) == 2 ? f<float, 2>(__VA_ARGS__)                                   \
                         : f<float, 1>(__VA_ARGS__)))


}  // namespace nrnn
