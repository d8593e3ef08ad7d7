// Dropout (and its gradient, the same map on dY): y = keep ? x * scale : 0,
// plus a residual.  The mask is drawn from the element's index by Philox and
// never stored, so the kernel moves its tensors once each and nothing else.
// Bound: HBM (x, the residual and y).
#include "ct_internal.h"
#include "philox.cuh"
#include "vec8.cuh"

namespace ct {

namespace {

template <typename T, bool RES>
__global__ void __launch_bounds__(256) dropout_kernel(const T *x, const T *residual, T *y, int64_t n,
                                                      RngArgs rng, bool vec) {
    const Philox philox(rng);
    const int64_t blocks = (n + 7) / 8;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < blocks;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t e = 8 * i;
        const uint32_t bits = n - e >= 8 ? 0xFFu : (1u << (int)(n - e)) - 1u;
        float v[8], r[8];
        load8(x + e, bits, vec, v);
        if (RES) load8(residual + e, bits, vec, r);
        const uint32_t keep = keep_bits(philox((uint64_t)i), rng.threshold);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = (keep >> k) & 1u ? v[k] * rng.scale : 0.f;
            if (RES) v[k] += r[k];
        }
        store8(y + e, bits, vec, v);
    }
}

template <typename T>
ct_status run(const void *x, const void *residual, void *y, int64_t n, const RngArgs &rng, cudaStream_t st) {
    const bool vec = (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)y) & 15) == 0;
    const int64_t want = ceil_div(ceil_div(n, 8), 256);
    const int grid = (int)(want < 148 * 16 ? want : 148 * 16);
    if (residual)
        dropout_kernel<T, true><<<grid, 256, 0, st>>>((const T *)x, (const T *)residual, (T *)y, n, rng, vec);
    else
        dropout_kernel<T, false><<<grid, 256, 0, st>>>((const T *)x, nullptr, (T *)y, n, rng, vec);
    return launch_status();
}

}  // namespace

ct_status dropout_run(int dtype, const void *x, const void *residual, void *y, int64_t n, const RngArgs &rng,
                      cudaStream_t st) {
    if (dtype == CT_F32) return run<float>(x, residual, y, n, rng, st);
    if (dtype == CT_F16) return run<__half>(x, residual, y, n, rng, st);
    return run<__nv_bfloat16>(x, residual, y, n, rng, st);
}

}  // namespace ct
