// Eight neighbouring elements of a tensor as floats: 32 bytes of fp32 (one
// 256-bit access, which sm_100 has), 16 of a 16-bit type.  The type is a value
// here, the same for a whole warp.
#pragma once

#include "ct_internal.h"
#include "vec16.cuh"

namespace ct {

__device__ __forceinline__ void load8_f32(const float *p, float (&f)[8]) {
    asm("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
        : "l"(p)
        : "memory");
}
__device__ __forceinline__ void store8_f32(float *p, const float (&f)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :
                 : "l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void load8_16(const T *p, float (&f)[8]) {
    float2 v[4];
    unpack(*reinterpret_cast<const uint4 *>(p), v, T());
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = v[j].x, f[2 * j + 1] = v[j].y;
}
template <typename T>
__device__ __forceinline__ void store8_16(T *p, const float (&f)[8]) {
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float2(f[2 * j], f[2 * j + 1]);
    *reinterpret_cast<uint4 *>(p) = pack(v, T());
}
template <typename T>
__device__ __forceinline__ void load_first(const T *p, int n, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < n ? to_f<T>(p[j]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_first(T *p, int n, const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = from_f<T>(f[j]);
}

// Elements e to e + 7 of a tensor, those from n on (n in 0..8 of them are the
// caller's) read as 0 and are not touched; vec: e's address is a vector's.
__device__ __forceinline__ void load8(const void *t, uint32_t dtype, int64_t e, int n, bool vec, float (&f)[8]) {
    vec = vec && n == 8;
    if (dtype == CT_F32) {
        if (vec) load8_f32((const float *)t + e, f);
        else load_first((const float *)t + e, n, f);
    } else if (dtype == CT_F16) {
        if (vec) load8_16((const __half *)t + e, f);
        else load_first((const __half *)t + e, n, f);
    } else {
        if (vec) load8_16((const __nv_bfloat16 *)t + e, f);
        else load_first((const __nv_bfloat16 *)t + e, n, f);
    }
}
__device__ __forceinline__ void store8(void *t, uint32_t dtype, int64_t e, int n, bool vec, const float (&f)[8]) {
    vec = vec && n == 8;
    if (dtype == CT_F32) {
        if (vec) store8_f32((float *)t + e, f);
        else store_first((float *)t + e, n, f);
    } else if (dtype == CT_F16) {
        if (vec) store8_16((__half *)t + e, f);
        else store_first((__half *)t + e, n, f);
    } else {
        if (vec) store8_16((__nv_bfloat16 *)t + e, f);
        else store_first((__nv_bfloat16 *)t + e, n, f);
    }
}

}  // namespace ct
