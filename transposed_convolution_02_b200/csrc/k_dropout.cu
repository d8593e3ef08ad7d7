// Dropout (and its gradient, the same map on dY): y = keep ? x * scale : 0,
// plus a residual.  The mask is drawn from the element's index by Philox and
// never stored, so the kernel moves its tensors once each and nothing else.
// Bound: HBM (x, the residual and y).
#include "ct_internal.h"
#include "philox.cuh"
#include "vec16.cuh"

namespace ct {

namespace {

#ifndef CT_DROP_U
#define CT_DROP_U 4
#endif
#ifndef CT_DROP_B
#define CT_DROP_B 4
#endif
#ifndef CT_DROP_G
#define CT_DROP_G (1 << 20)
#endif
constexpr int kThreads = 256;
constexpr int kUnroll = CT_DROP_U;   // blocks of the generator that a thread has in flight

// A thread takes eight elements, one block of the generator, at a time.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads, CT_DROP_B) dropout_kernel(const T *x, const T *residual, T *y, int64_t n,
                                                                      const __grid_constant__ RngArgs rng, bool vec) {
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
    if (vec) {
        for (; i < blocks; i += kUnroll * stride) {
            uint4 a[kUnroll][Q], b[kUnroll][Q];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (i + u * stride < blocks)
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        a[u][q] = *reinterpret_cast<const uint4 *>(x + 8 * (i + u * stride) + q * V);
                        if (RES) b[u][q] = *reinterpret_cast<const uint4 *>(residual + 8 * (i + u * stride) + q * V);
                    }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (i + u * stride < blocks) {
                    const uint4 d = philox((uint64_t)(i + u * stride));
                    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        float2 v[P], r[P] = {};
                        unpack(a[u][q], v, T());
                        if (RES) unpack(b[u][q], r, T());
                        one(v, w + q * P, r);
                        *reinterpret_cast<uint4 *>(y + 8 * (i + u * stride) + q * V) = pack(v, T());
                    }
                }
        }
    } else {
        for (; i < blocks; i += stride) {
            const uint4 d = philox((uint64_t)i);
            const uint32_t w[4] = {d.x, d.y, d.z, d.w};
            float2 v[Q][P], r[Q][P] = {};
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                unpack(gather(x + 8 * i + q * V), v[q], T());
                if (RES) unpack(gather(residual + 8 * i + q * V), r[q], T());
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                one(v[q], w + q * P, r[q]);
                store_some(y + 8 * i + q * V, ~0u, v[q]);
            }
        }
    }
    if ((n & 7) != 0 && blockIdx.x == 0 && threadIdx.x == 0) {   // the last elements
        i = blocks;
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
    const int64_t want = ceil_div(ceil_div(n, 8), (int64_t)kThreads * kUnroll);
    const int grid = (int)(want < 1 ? 1 : want < CT_DROP_G ? want : CT_DROP_G);
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
