// Eight neighbouring elements of a tensor as floats: 32 bytes of fp32 (one
// 256-bit access, which sm_100 has), 16 of a 16-bit type.  The type is a value
// here, the same for a whole warp.
#pragma once

#include "ct_internal.h"
#include "vec16.cuh"

namespace ct {

__device__ __forceinline__ void load8_f32(const float *p, float2 (&f)[4]) {
    asm("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(f[0].x), "=f"(f[0].y), "=f"(f[1].x), "=f"(f[1].y), "=f"(f[2].x), "=f"(f[2].y), "=f"(f[3].x), "=f"(f[3].y)
        : "l"(p)
        : "memory");
}
__device__ __forceinline__ void store8_f32(float *p, const float2 (&f)[4]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :
                 : "l"(p), "f"(f[0].x), "f"(f[0].y), "f"(f[1].x), "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x),
                   "f"(f[3].y)
                 : "memory");
}

// The first n of the eight.
template <typename T>
__device__ __forceinline__ void load_first(const T *p, int n, float2 (&f)[4]) {
    load_some(p, (1u << n) - 1u, f);
}
template <typename T>
__device__ __forceinline__ void store_first(T *p, int n, const float2 (&f)[4]) {
    store_some(p, (1u << n) - 1u, f);
}
template <typename T>
__device__ __forceinline__ void load8_16(const T *p, float2 (&f)[4]) {
    unpack(*reinterpret_cast<const uint4 *>(p), f, T());
}
template <typename T>
__device__ __forceinline__ void store8_16(T *p, const float2 (&f)[4]) {
    *reinterpret_cast<uint4 *>(p) = pack(f, T());
}

// Elements e to e + 7 of a tensor, those from n on (n in 0..8 of them are the
// caller's) read as 0 and are not touched; vec: e's address is a vector's.
__device__ __forceinline__ void load8(const void *t, uint32_t dtype, int64_t e, int n, bool vec, float2 (&f)[4]) {
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
__device__ __forceinline__ void store8(void *t, uint32_t dtype, int64_t e, int n, bool vec, const float2 (&f)[4]) {
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
