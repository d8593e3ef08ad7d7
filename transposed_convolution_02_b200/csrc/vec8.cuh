// Eight neighbouring elements of a tensor as eight floats: 16 bytes of a
// 16-bit type, 32 of fp32.  `bits` marks the elements that belong to the
// caller; the full mask on 16-byte aligned tensors moves whole vectors.
// Conversions to 16 bits round once, to nearest even.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ct {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float2 pair_to_f(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 pair_to_f(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pair_from_f(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pair_from_f(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The raw words of a vector, so that several loads can be in flight before
// the first is converted.
template <typename T>
struct Vec8 {
    uint4 w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float v[8]) const {
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = pair_to_f(q[j], T());
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store(T *p, const float v[8]) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pair_from_f(v[0], v[1], T()), pair_from_f(v[2], v[3], T()),
                       pair_from_f(v[4], v[5], T()), pair_from_f(v[6], v[7], T()));
    }
};

template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float v[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float v[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// Elements outside `bits` read as 0 and are neither read nor written.
template <typename T>
__device__ __forceinline__ void load8(const T *p, uint32_t bits, bool vec, float v[8]) {
    if (vec && bits == 0xFFu) {
        Vec8<T> r;
        r.load(p);
        r.get(v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (bits >> k) & 1u ? to_f<T>(p[k]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, uint32_t bits, bool vec, const float v[8]) {
    if (vec && bits == 0xFFu) {
        Vec8<T>::store(p, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if ((bits >> k) & 1u) p[k] = from_f<T>(v[k]);
    }
}

}  // namespace ct
