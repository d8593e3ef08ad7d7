// Dropout (and its gradient, the same map on dY): y = keep ? x * scale : 0,
// plus a residual.  The mask is drawn from the element's index by Philox and
// never stored, so the kernel moves its tensors once each and nothing else.
// Bound: HBM (x, the residual and y), with the generator near it: ten rounds
// for eight elements.  What counts is loads in flight: four vectors
// of each tensor per thread at 1024 threads an SM, every thread done after them.
// 33.5M bf16 with a residual (201 MB) 32 us, 0.96 of the measured copy rate (one
// vector in flight 49 us, two 34); 33.5M fp16 without (134 MB) 25.5 us, 0.80
// (one 34 us; 27.9 with the round keys added up on the way).
#include "ct_internal.h"
#include "philox.cuh"
#include "vec16.cuh"

namespace ct {

namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 4;             // of a tensor, that a thread has in flight
constexpr int kBlocksPerSm = 4;
constexpr int64_t kMaxGrid = 1 << 20;

// A thread takes eight elements, one block of the generator, at a time.
template <typename T, bool RES, bool FIXED>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    dropout_kernel(const T *x, const T *residual, T *y, int64_t n, const __grid_constant__ RngArgs rng, bool vec) {
    constexpr int V = kVec<T>, P = V / 2, Q = 8 / V, U = kVectors / Q;   // vectors of P pairs, Q to a block
    const Philox<FIXED> philox(rng);
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
        for (; i < blocks; i += U * stride) {
            uint4 a[U][Q], b[U][Q];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * stride < blocks)
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        a[u][q] = *reinterpret_cast<const uint4 *>(x + 8 * (i + u * stride) + q * V);
                        if (RES) b[u][q] = *reinterpret_cast<const uint4 *>(residual + 8 * (i + u * stride) + q * V);
                    }
#pragma unroll
            for (int u = 0; u < U; ++u)
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
    const int64_t want = ceil_div(ceil_div(n, 8), (int64_t)kThreads * kVectors * kVec<T> / 8);
    const int grid = (int)(want < 1 ? 1 : want < kMaxGrid ? want : kMaxGrid);
    auto launch = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, st>>>((const T *)x, (const T *)residual, (T *)y, n, rng, vec);
    };
    if (residual) {
        if (rng.dev) launch(dropout_kernel<T, true, false>);
        else launch(dropout_kernel<T, true, true>);
    } else {
        if (rng.dev) launch(dropout_kernel<T, false, false>);
        else launch(dropout_kernel<T, false, true>);
    }
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
