// e4m3 codes with an fp32 scale for a block of them: code * scale is the value.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace ct {

constexpr float kE4m3Max = 448.f;
// The least scale: its reciprocal is finite, and a block of zeros has one.
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126

// Where one of the two is NaN, so is the result (fmaxf drops it): a block that
// holds a NaN gets a scale of NaN, and so shows it whatever its codes are.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest magnitude of three, NaN likewise.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float scale_of(float amax) { return max_nan(amax * (1.f / kE4m3Max), kLeastScale); }

// Two codes, to nearest even, at most 448 in magnitude (x in the low byte).
__device__ __forceinline__ uint32_t codes2(float x, float y) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    return codes2(a, b) | codes2(c, d) << 16;
}

}  // namespace ct
