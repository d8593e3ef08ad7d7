// Sixteen bytes of a tensor as floats: eight neighbours of a 16-bit type,
// four of fp32.  `bits` marks the elements that belong to the caller; the full
// mask on 16-byte aligned tensors moves whole vectors.  Conversions to 16 bits
// round once, to nearest even.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ct {

template <typename T>
constexpr int kVec = 16 / sizeof(T);

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

// The words of a vector as pairs of floats, and back.
__device__ __forceinline__ void unpack(uint4 w, float2 (&v)[2], float) {
    v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
}
__device__ __forceinline__ float2 unpack1(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 unpack1(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ void unpack(uint4 w, float2 (&v)[4], T) {
    v[0] = unpack1(w.x, T());
    v[1] = unpack1(w.y, T());
    v[2] = unpack1(w.z, T());
    v[3] = unpack1(w.w, T());
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[2], float) {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                      __float_as_uint(v[1].y));
}
__device__ __forceinline__ uint32_t pack1(float2 a, __half) {
    const __half2 h = __floats2half2_rn(a.x, a.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack1(float2 a, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float2 (&v)[4], T) {
    return make_uint4(pack1(v[0], T()), pack1(v[1], T()), pack1(v[2], T()), pack1(v[3], T()));
}

// Element by element the smaller and the larger of two vectors.
__device__ __forceinline__ uint32_t smaller1(uint32_t a, uint32_t b, float) {
    return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t larger1(uint32_t a, uint32_t b, float) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t smaller1(uint32_t a, uint32_t b, __half) {
    const __half2 m = __hmin2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
__device__ __forceinline__ uint32_t larger1(uint32_t a, uint32_t b, __half) {
    const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
__device__ __forceinline__ uint32_t smaller1(uint32_t a, uint32_t b, __nv_bfloat16) {
    const __nv_bfloat162 m =
        __hmin2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
__device__ __forceinline__ uint32_t larger1(uint32_t a, uint32_t b, __nv_bfloat16) {
    const __nv_bfloat162 m =
        __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
template <typename T>
__device__ __forceinline__ uint4 smaller(uint4 a, uint4 b, T t) {
    return make_uint4(smaller1(a.x, b.x, t), smaller1(a.y, b.y, t), smaller1(a.z, b.z, t), smaller1(a.w, b.w, t));
}
template <typename T>
__device__ __forceinline__ uint4 larger(uint4 a, uint4 b, T t) {
    return make_uint4(larger1(a.x, b.x, t), larger1(a.y, b.y, t), larger1(a.z, b.z, t), larger1(a.w, b.w, t));
}

// A vector from any element's address.
__device__ __forceinline__ uint4 gather(const float *p) {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
    return make_uint4(q[0], q[1], q[2], q[3]);
}
template <typename T>
__device__ __forceinline__ uint4 gather(const T *p) {
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
    return make_uint4(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16, q[4] | (uint32_t)q[5] << 16,
                      q[6] | (uint32_t)q[7] << 16);
}

// Elements outside `bits` read as 0 and are neither read nor written.
template <typename T, int P>
__device__ __forceinline__ void load_some(const T *p, uint32_t bits, float2 (&v)[P]) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
        v[j].x = (bits >> (2 * j)) & 1u ? to_f<T>(p[2 * j]) : 0.f;
        v[j].y = (bits >> (2 * j + 1)) & 1u ? to_f<T>(p[2 * j + 1]) : 0.f;
    }
}

template <typename T, int P>
__device__ __forceinline__ void store_some(T *p, uint32_t bits, const float2 (&v)[P]) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
        if ((bits >> (2 * j)) & 1u) p[2 * j] = from_f<T>(v[j].x);
        if ((bits >> (2 * j + 1)) & 1u) p[2 * j + 1] = from_f<T>(v[j].y);
    }
}

template <typename T, int P>
__device__ __forceinline__ void store_vec(T *p, bool vec, const float2 (&v)[P]) {
    if (vec) *reinterpret_cast<uint4 *>(p) = pack(v, T());
    else store_some(p, ~0u, v);
}

template <typename T, int P>
__device__ __forceinline__ void load_vec(const T *p, bool vec, float2 (&v)[P]) {
    unpack(vec ? *reinterpret_cast<const uint4 *>(p) : gather(p), v, T());
}

}  // namespace ct
