// Dropout (and its gradient, the same map on dY): y = keep ? x * scale : 0,
// plus a residual.  The mask is drawn from the element's index by Philox and
// never stored, so the kernel moves its tensors once each and nothing else.
// Bound: HBM (x, the residual and y).
#include "ct_internal.h"
#include "philox.cuh"
#include "vec16.cuh"

namespace ct {

namespace {

constexpr int kThreads = 256;

// A thread takes eight elements, one block of the generator, at a time.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const T *x, const T *residual, T *y, int64_t n,
                                                           RngArgs rng, bool vec) {
    constexpr int V = kVec<T>, P = V / 2, Q = 8 / V;   // vectors of P pairs, Q to a block
    const Philox philox(rng);
    const uint32_t limit = drop_limit(rng.threshold);
    const bool all = rng.threshold == 0;
    auto one = [&](float2 (&v)[P], const uint32_t *w, const float2 (&r)[P]) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if (!all) v[j] = drop_pair(w[j], limit, rng.scale, v[j]);
            if (RES) v[j] = __fadd2_rn(v[j], r[j]);
        }
    };
    const int64_t blocks = n / 8, stride = (int64_t)gridDim.x * kThreads;
    int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    for (; i < blocks; i += stride) {
        float2 v[Q][P], r[Q][P] = {};
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            load_vec(x + 8 * i + q * V, vec, v[q]);
            if (RES) load_vec(residual + 8 * i + q * V, vec, r[q]);
        }
        const uint4 d = philox((uint64_t)i);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            one(v[q], w + q * P, r[q]);
            store_vec(y + 8 * i + q * V, vec, v[q]);
        }
    }
    if (i == blocks && (n & 7)) {   // the last elements
        const uint4 d = philox((uint64_t)i);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
        const uint32_t bits = (1u << (n & 7)) - 1u;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float2 v[P], r[P] = {};
            load_some(x + 8 * i + q * V, bits >> (q * V), v);
            if (RES) load_some(residual + 8 * i + q * V, bits >> (q * V), r);
            one(v, w + q * P, r);
            store_some(y + 8 * i + q * V, bits >> (q * V), v);
        }
    }
}

template <typename T>
ct_status run(const void *x, const void *residual, void *y, int64_t n, const RngArgs &rng, cudaStream_t st) {
    const bool vec = (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)y) & 15) == 0;
    const int64_t want = ceil_div(ceil_div(n, 8), kThreads);
    const int grid = (int)(want < 148 * 8 ? want : 148 * 8);
    if (residual)
        dropout_kernel<T, true><<<grid, kThreads, 0, st>>>((const T *)x, (const T *)residual, (T *)y, n, rng, vec);
    else
        dropout_kernel<T, false><<<grid, kThreads, 0, st>>>((const T *)x, nullptr, (T *)y, n, rng, vec);
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
