// experts_common.hpp -- shared pieces of the expert-layer kernels: element
// types, argument checks and the device status. Part of libpca_hist.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "experts.h"
#include "hist_host.hpp"

namespace pca_experts {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t s32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <class T> struct Vec8;
template <> struct Vec8<__bf16> { typedef bf16x8 type; };
template <> struct Vec8<_Float16> { typedef f16x8 type; };

// Loads and stores of 16 (or 8) bytes at any address: the compiler emits one
// wide access, which gfx950 takes at byte alignment.
template <class V>
__device__ __forceinline__ V load_any(const void *p)
{
    V v;
    __builtin_memcpy(&v, p, sizeof(V));
    return v;
}

template <class V>
__device__ __forceinline__ void store_any(void *p, V v)
{
    __builtin_memcpy(p, &v, sizeof(V));
}

// Eight elements from p, of which `left` lie in the row (the others read 0).
template <class T>
__device__ __forceinline__ typename Vec8<T>::type load8(const T *p, int left)
{
    if (left >= 8) return load_any<typename Vec8<T>::type>(p);
    typename Vec8<T>::type v = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) v[i] = p[i];
    return v;
}

template <class T>
__device__ __forceinline__ void store8(T *p, typename Vec8<T>::type v, int left)
{
    if (left >= 8) {
        store_any(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = v[i];
}

typedef int8_t i8x8 __attribute__((ext_vector_type(8)));

// f / scale to the nearest whole number, ties to even, for |f| up to 127 scale (scale > 0). The quotient
// by the reciprocal is within 127 * 2^-23 = 0.000015 of the real one, so its rounding is right unless it lies
// that near a half; only eights with such a value, and scales that have no normal reciprocal, take the way
// that decides exactly (taken for every value, quantising was bound by its arithmetic: 8192 x 4096 in 30 us, not 28).
struct Steps {
    float scale, inverse;
    bool normal;
    explicit __device__ __forceinline__ Steps(float scale)
        : scale(scale), normal(scale > 1e-37f && scale < 1e37f)
    {
        inverse = normal ? 1.0f / scale : 0.f;
    }
    __device__ __forceinline__ i8x8 operator()(const float (&f)[8]) const
    {
        float n[8], most = normal ? 0.f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = f[i] * inverse;
            n[i] = rintf(t);
            most = fmaxf(most, fabsf(t - n[i]));
        }
        if (most > 0.49998f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float m = rintf(f[i] / scale);
                // What m leaves of f is exact in 32 bits: a multiple of the last bit of scale (or of f, if that
                // is less than scale, and m 0 or 1), and no more than some half of scale. Comparing it with
                // half the scale decides.
                const float rest = __builtin_fmaf(-m, scale, f[i]);
                const float twice = 2.f * fabsf(rest);
                const bool odd = ((int)m & 1) != 0;
                if (twice > scale || (twice == scale && odd)) m += rest > 0.f ? 1.f : -1.f;
                n[i] = fminf(fmaxf(m, -127.f), 127.f);
            }
        }
        i8x8 q;
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = (int8_t)(int)n[i];
        return q;
    }
};

// Eight 8-bit values to p, of which `left` lie in the row.
__device__ __forceinline__ void store8(int8_t *p, i8x8 v, int left)
{
    if (left >= 8) {
        store_any(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = v[i];
}

__device__ __forceinline__ void lds_add(uint32_t *lds, uint32_t slot, uint32_t v)
{
    __hip_atomic_fetch_add(lds + slot, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// Inclusive sum over the wave's lanes, all of them active: within rows of 16
// lanes by row shifts, then lane 15 of each row into the next and lane 31 into
// the upper half (DPP, no LDS round trip).
__device__ __forceinline__ uint32_t wave_inclusive_scan(uint32_t v)
{
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, true);   // row_shr:1
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, true);   // row_shr:2
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, true);   // row_shr:4
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, true);   // row_shr:8
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false);  // row_bcast:15
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false);  // row_bcast:31
    return v;
}

__device__ __forceinline__ float wave_sum_f(float v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// The current device's status (gfx950 or not).
inline hist_status_t device_status()
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return HIST_ERR_UNSUPPORTED;
    }
    return pca_host::device_supported(dev);
}

// What one launch takes at `each` a workgroup: it is limited to 2^32 - 1 threads. The operators whose
// rows are their own work queue as many launches as that needs.
inline uint64_t most_of(uint64_t each, uint32_t threads) { return UINT32_MAX / threads * each; }

// Queues a kernel.
template <class... P, class... A>
hist_status_t launch(void (*kernel)(P...), uint64_t blocks, uint32_t threads, uint32_t lds,
                     hipStream_t stream, A... args)
{
    if (blocks > UINT32_MAX / threads) return HIST_ERR_UNSUPPORTED;
    if (blocks == 0) return HIST_OK;
    if (lds > 65536 && hipFuncSetAttribute((const void *)kernel,
                                           hipFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)lds) != hipSuccess) {
        (void)hipGetLastError();
        return HIST_ERR_HIP;
    }
    kernel<<<(uint32_t)blocks, threads, lds, stream>>>(((P)args)...);
    return hipGetLastError() == hipSuccess ? HIST_OK : HIST_ERR_HIP;
}

inline bool dtype_ok(int32_t dtype) { return dtype == EXPERTS_BF16 || dtype == EXPERTS_FP16; }
inline bool misaligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

}  // namespace pca_experts
