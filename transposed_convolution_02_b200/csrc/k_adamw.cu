// AdamW (Loshchilov and Hutter, "Decoupled weight decay regularization", 2019)
// over many tensors in one launch, and the global norm of their gradients:
//
//     g' = g * scale,   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//     p  = p - lr (wd p + m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps))
//
// Bound: HBM; 28 bytes an element in fp32, 16 with 8-bit states, against some
// 20 operations, 80 with 8-bit states.  Warps take blocks of 256 elements,
// eight neighbours a lane, so that each tensor's part is one access.
//
// 8-bit states.  A block holds its m, and the square roots of its v (half the
// exponents), as e4m3 codes under an fp32 scale each, largest magnitude / 448.
// Their steps are 6 to 12% of a value, its decay in one update 0.1% (v) or 10%
// (m): rounding to nearest would keep v for good.  Rounding is therefore
// random and right on average: up with the probability of the part that lies
// beyond the lower code.  The bits are 16 of Philox for an element (its place
// in the states), a seed and the step, the same for m and v.  A root above 0
// becomes no code of 0, which would divide m by eps.
#include <math.h>

#include "adamw.h"
#include "ct_cuda_util.h"
#include "e4m3.cuh"
#include "sm100.cuh"
#include "vec32.cuh"

namespace ct {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr float kLow = 0.015625f;        // 2^-6: below it codes lie 2^-9 apart
constexpr float kLeastCode = 0.001953125f;   // 2^-9

template <int N>
__device__ __forceinline__ int find(const TensorTable<N> &table, int64_t block) {
    int lo = 0, hi = table.count - 1;         // the last entry that starts at or before the block
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (table.t[mid].first <= block) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// x to e4m3's grid, up or down as 16 random bits say: they are added where the
// mantissa's three bits end, and what lies below those is cut off.  (The 4 bits
// below the random ones are dropped: 2^-16 of a step.)  Below 2^-6 values are
// moved to where codes lie as far apart.  NaN stays; what passes 448 is cut by
// the conversion.
__device__ __forceinline__ float to_grid(float x, uint32_t random) {
    const float a = fabsf(x);
    const bool low = a < kLow;
    float b = low ? a + kLow : a;
    b = __uint_as_float((__float_as_uint(b) + (random << 4)) & ~0xFFFFFu);
    b = low ? b - kLow : b;
    return copysignf(b, x);
}

// a / b from b's rounded reciprocal, corrected by the remainder: correctly
// rounded (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990) where nothing underflows; two operations more
// than the product, where a division would take ten.
__device__ __forceinline__ float quotient(float a, float b, float reciprocal) {
    const float q = a * reciprocal;
    return fmaf(fmaf(-q, b, a), reciprocal, q);
}

__device__ __forceinline__ void from_codes(uint2 w, float scale, float (&f)[8]) {
    const uint32_t word[2] = {w.x, w.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(word[j / 2] >> (16 * (j & 1)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        f[2 * j] = v.x * scale;
        f[2 * j + 1] = v.y * scale;
    }
}

// The scale of a warp's 256 values (magnitudes compare as whole numbers, NaN
// above all) and its reciprocal.
__device__ __forceinline__ float warp_scale(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    return scale_of(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, m)));
}

struct Step {
    float lr, lr_c1, root_c2;
};

__device__ __forceinline__ Step step_of(const AdamWParams &p, uint64_t t) {
    Step s = {p.lr, p.lr_c1, p.root_c2};
    if (p.lr_dev || p.step_dev) {
        const float lr = p.lr_dev ? *p.lr_dev : p.lr;
        // 1 - b^t without a cancellation where t log b is small
        s = {lr, lr / -expm1f((float)t * p.log1), rsqrtf(-expm1f((float)t * p.log2))};
    }
    return s;
}

template <int BITS, int N>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ TensorTable<N> table, const __grid_constant__ AdamWParams p, int per) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t block = (int64_t)blockIdx.x * kWarps * per + warp;
    if (block >= table.blocks) return;
    const float gs = p.grad_scale ? *p.grad_scale : 1.f;
    if (!(gs > 0.f && gs <= 3.4028234e38f)) return;      // nothing is touched
    const uint64_t t = p.step_dev ? (uint64_t)*p.step_dev : p.step;
    const Step s = step_of(p, t);
    int i = find(table, block);
    for (int k = 0; k < per && block < table.blocks; ++k, block += kWarps) {
        while (i + 1 < table.count && table.t[i + 1].first <= block) ++i;
        const TensorEntry &e = table.t[i];
        const int64_t at = (block - e.first) * kBlock + lane * 8;       // in the tensor
        const int64_t in = e.state + (block - e.first);                 // block of the states
        const int n = e.n - at >= 8 ? 8 : e.n > at ? (int)(e.n - at) : 0;
        const uint32_t pd = e.kind & 3, gd = (e.kind >> 2) & 3;
        float *master = pd != CT_F32 ? p.master + (e.master + block - e.first) * kBlock + lane * 8 : nullptr;
        float g[8], w[8], m[8], v[8];
        load8(e.grad, gd, at, n, e.kind & kGradVec, g);
        if (master) load8_f32(master, w);
        else load8(e.param, CT_F32, at, n, e.kind & kParamVec, w);
        if (BITS == 32) {
            load8_f32((const float *)p.m + in * kBlock + lane * 8, m);
            load8_f32((const float *)p.v + in * kBlock + lane * 8, v);
        } else {
            const uint2 cm = *reinterpret_cast<const uint2 *>((const uint8_t *)p.m + in * kBlock + lane * 8);
            const uint2 cv = *reinterpret_cast<const uint2 *>((const uint8_t *)p.v + in * kBlock + lane * 8);
            from_codes(cm, p.m_scale[in], m);
            from_codes(cv, p.v_scale[in], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= v[j];
        }
        if (n < 8) {         // what lies behind the tensor in its last block counts for nothing, and becomes 0
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= n) w[j] = m[j] = v[j] = 0.f;
        }
        const float lr_wd = s.lr * e.decay;
        float root[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // each operation rounded, as the formulas stand: what 8-bit codes are
            // chosen by is then the same wherever it is computed in fp32
            const float a = g[j] * gs;
            m[j] = __fadd_rn(__fmul_rn(p.beta1, m[j]), __fmul_rn(p.rest1, a));
            v[j] = __fadd_rn(__fmul_rn(p.beta2, v[j]), __fmul_rn(p.rest2, __fmul_rn(a, a)));
            if (BITS == 8) root[j] = __fsqrt_rn(v[j]);
            else asm("sqrt.approx.f32 %0, %1;" : "=f"(root[j]) : "f"(v[j]));     // to 2^-23
            w[j] -= fmaf(lr_wd, w[j], s.lr_c1 * __fdividef(m[j], fmaf(root[j], s.root_c2, p.eps)));
        }
        if (master) {
            store8_f32(master, w);
            store8(e.param, pd, at, n, e.kind & kParamVec, w);
        } else {
            store8(e.param, CT_F32, at, n, e.kind & kParamVec, w);
        }
        if (BITS == 32) {
            store8_f32((float *)p.m + in * kBlock + lane * 8, m);
            store8_f32((float *)p.v + in * kBlock + lane * 8, v);
        } else {
            const float sm = warp_scale(m), sv = warp_scale(root);
            const float im = 1.f / sm, iv = 1.f / sv;
            Philox<true> philox(p.rng);
            philox.c2 = (uint32_t)t;
            philox.c3 = (uint32_t)(t >> 32);
            const uint4 d = philox((uint64_t)(in * (kBlock / 8) + lane));
            const uint32_t bits[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t r = j & 1 ? bits[j / 2] >> 16 : bits[j / 2] & 0xFFFFu;
                m[j] = to_grid(quotient(m[j], sm, im), r);
                const float c = to_grid(quotient(root[j], sv, iv), r);
                v[j] = root[j] > 0.f ? fmaxf(c, kLeastCode) : c;
            }
            *reinterpret_cast<uint2 *>((uint8_t *)p.m + in * kBlock + lane * 8) =
                make_uint2(codes4(m[0], m[1], m[2], m[3]), codes4(m[4], m[5], m[6], m[7]));
            *reinterpret_cast<uint2 *>((uint8_t *)p.v + in * kBlock + lane * 8) =
                make_uint2(codes4(v[0], v[1], v[2], v[3]), codes4(v[4], v[5], v[6], v[7]));
            if (lane == 0) {
                p.m_scale[in] = sm;
                p.v_scale[in] = sv;
            }
        }
    }
}

// ---- the gradients' norm ------------------------------------------------------

// Squares and sums of eight in fp32, from there on in 64 bits: a step has
// billions of them.  A thread block has a run of blocks; its order and that of
// the join depend on sizes alone.
template <int N>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ TensorTable<N> table, double *partial) {
    __shared__ double side[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t each = (table.blocks + gridDim.x - 1) / gridDim.x;
    const int64_t first = blockIdx.x * each, last = first + each < table.blocks ? first + each : table.blocks;
    double sum = 0.0;
    if (first + warp < last) {
        int i = find(table, first + warp);
        for (int64_t block = first + warp; block < last; block += kWarps) {
            while (i + 1 < table.count && table.t[i + 1].first <= block) ++i;
            const TensorEntry &e = table.t[i];
            const int64_t at = (block - e.first) * kBlock + lane * 8;
            const int n = e.n - at >= 8 ? 8 : e.n > at ? (int)(e.n - at) : 0;
            float g[8], q = 0.f;
            load8(e.grad, (e.kind >> 2) & 3, at, n, e.kind & kGradVec, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) q = fmaf(g[j], g[j], q);
            sum += (double)q;
        }
    }
    for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) side[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) sum += side[w];
        partial[blockIdx.x] = sum;
    }
}

__global__ void __launch_bounds__(kThreads)
    norm_join_kernel(const double *partial, int64_t n, double max_norm, float *norm, float *scale) {
    __shared__ double side[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double sum = 0.0;
    sm100::griddep_wait();
    for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += partial[i];
    for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) side[warp] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < kWarps; ++w) sum += side[w];
    const double root = sqrt(sum);
    *norm = (float)root;
    // a norm that fp32 does not hold is no norm to scale by
    const bool finite = (float)root <= 3.4028234e38f;
    if (scale) *scale = !finite ? 0.f : root > max_norm ? (float)(max_norm / root) : 1.f;
}

// ---- host ---------------------------------------------------------------------

bool on_vector(const void *p, int dtype) { return ((uintptr_t)p & (dtype == CT_F32 ? 31 : 15)) == 0; }

// Tables of the tensors that have a gradient and an element, in order:
// launch(table) for each.
template <int N, typename F>
ct_status by_table(int64_t count, const ct_param *shapes, void *const *params, const void *const *grads, F launch) {
    TensorTable<N> table;
    table.count = 0;
    table.blocks = 0;
    int64_t state = 0, master = 0;
    for (int64_t i = 0; i < count; ++i) {
        const ct_param &s = shapes[i];
        const int64_t blocks = ceil_div(s.n, (int64_t)kBlock);
        if (blocks > 0 && grads[i]) {
            TensorEntry &e = table.t[table.count++];
            e.param = params ? params[i] : nullptr;
            e.grad = grads[i];
            e.n = s.n;
            e.first = table.blocks;
            e.state = state;
            e.master = master;
            e.decay = (float)s.weight_decay;
            e.kind = (uint32_t)s.dtype | (uint32_t)s.grad_dtype << 2 | (on_vector(e.param, s.dtype) ? kParamVec : 0) |
                     (on_vector(e.grad, s.grad_dtype) ? kGradVec : 0);
            table.blocks += blocks;
            if (table.count == N) {
                const ct_status st = launch(table);
                if (st != CT_OK) return st;
                table.count = 0;
                table.blocks = 0;
            }
        }
        state += blocks;
        if (s.dtype != CT_F32) master += blocks;
    }
    return table.count > 0 ? launch(table) : CT_OK;
}

template <int BITS, int N>
ct_status adamw_tables(int64_t count, const ct_param *shapes, void *const *params, const void *const *grads,
                       const AdamWParams &p, cudaStream_t st) {
    return by_table<N>(count, shapes, params, grads, [&](const TensorTable<N> &table) {
        // up to four blocks a warp, where that leaves four thread blocks an SM
        int64_t per = table.blocks / (148 * 4 * kWarps);
        per = per < 1 ? 1 : per > 4 ? 4 : per;
        int64_t grid = ceil_div(table.blocks, per * kWarps);
        if (grid > 0x7FFFFFFF) return CT_ERR_ATTR;
        adamw_kernel<BITS, N><<<(unsigned)grid, kThreads, 0, st>>>(table, p, (int)per);
        return launch_status();
    });
}

template <int N>
ct_status norm_tables(int64_t count, const ct_param *shapes, const void *const *grads, double max_norm, float *norm,
                      float *scale, double *ws, cudaStream_t st) {
    int64_t parts = 0;
    ct_status s = by_table<N>(count, shapes, nullptr, grads, [&](const TensorTable<N> &table) {
        const int64_t want = ceil_div(table.blocks, (int64_t)kWarps);
        const int64_t grid = want < kNormBlocks ? want : kNormBlocks;
        norm_kernel<N><<<(unsigned)grid, kThreads, 0, st>>>(table, ws + parts);
        parts += grid;
        return launch_status();
    });
    if (s != CT_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = parts > 0 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, norm_join_kernel, (const double *)ws, parts, max_norm, norm, scale) != cudaSuccess) {
        cudaGetLastError();
        return CT_ERR_DEVICE;
    }
    return CT_OK;
}

}  // namespace

ct_status adamw_run(const ct_adamw_desc *d, int64_t count, const ct_param *shapes, void *const *params,
                    const void *const *grads, AdamWParams &p, cudaStream_t st) {
    const double c1 = -expm1((double)d->step * log(d->beta1)), c2 = -expm1((double)d->step * log(d->beta2));
    p.beta1 = (float)d->beta1;
    p.beta2 = (float)d->beta2;
    p.rest1 = (float)(1.0 - d->beta1);
    p.rest2 = (float)(1.0 - d->beta2);
    p.eps = (float)d->eps;
    p.lr = (float)d->lr;
    p.lr_c1 = (float)(d->lr / c1);
    p.root_c2 = (float)(1.0 / sqrt(c2));
    p.log1 = (float)log(d->beta1);
    p.log2 = (float)log(d->beta2);
    p.step = (uint64_t)d->step;
    p.rng.seed = d->seed;
    set_keys(p.rng);
    if (d->bits == 32)
        return count <= kFewTensors ? adamw_tables<32, kFewTensors>(count, shapes, params, grads, p, st)
                                    : adamw_tables<32, kManyTensors>(count, shapes, params, grads, p, st);
    return count <= kFewTensors ? adamw_tables<8, kFewTensors>(count, shapes, params, grads, p, st)
                                : adamw_tables<8, kManyTensors>(count, shapes, params, grads, p, st);
}

ct_status grad_norm_run(int64_t count, const ct_param *shapes, const void *const *grads, double max_norm, float *norm,
                        float *scale, double *ws, cudaStream_t st) {
    return count <= kFewTensors ? norm_tables<kFewTensors>(count, shapes, grads, max_norm, norm, scale, ws, st)
                                : norm_tables<kManyTensors>(count, shapes, grads, max_norm, norm, scale, ws, st);
}

}  // namespace ct
