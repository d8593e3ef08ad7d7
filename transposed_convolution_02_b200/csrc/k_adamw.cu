// AdamW (Loshchilov and Hutter, "Decoupled weight decay regularization", 2019)
// over many tensors in one launch, and the global norm of their gradients:
//
//     g' = g * scale,   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//     p  = p - lr (wd p + m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps))
//
// Bound: HBM; 28 bytes an element in fp32, 16 with 8-bit states, against some
// 20 operations, 60 with 8-bit states.  Warps take blocks of 256 elements,
// eight neighbours a lane, so that each tensor's part is one access.
// Measured (GPU time; against the measured copy rate): 67M fp32 271 us (1.06),
// with 8-bit states 186 (0.89: instructions issue in 0.70 of the cycles).
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

#include <type_traits>

#include "adamw.h"
#include "ct_cuda_util.h"
#include "e4m3.cuh"
#include "sm100.cuh"
#include "vec32.cuh"

namespace ct {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

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

// The e4m3 code of |x| (at most 448), up or down as 16 random bits say, in
// bits 24 to 30.  x * 2^-120 has e4m3's exponents as its own, and its values
// below 2^-6 among fp32's numbers without one: its bits are the code from 20
// on, with the part that lies beyond it below.  Shifted up by 4 (the sign is
// gone), they take the random bits (8 to 23) and carry.  (The lowest 4 bits are
// dropped: 2^-16 of a step.)
__device__ __forceinline__ uint32_t code_of(float x, uint32_t random) {
    return min((__float_as_uint(x) << 4) + random, 0x7EFFFFFFu);
}
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// The sum of two floats each.  A product and a sum of two floats (__fmul2_rn,
// __fadd2_rn) become one operation, of one rounding, where they meet; these do
// not.
__device__ __forceinline__ float2 plus(float2 a, float2 b) {
    return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// a / b from b's rounded reciprocal, corrected by the remainder: correctly
// rounded (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990) where nothing underflows; two operations more
// than the product, where a division would take ten.
__device__ __forceinline__ float2 quotient(float2 a, float minus_b, float reciprocal) {
    const float2 r = make_float2(reciprocal, reciprocal), q = __fmul2_rn(a, r);
    return __ffma2_rn(__ffma2_rn(q, make_float2(minus_b, minus_b), a), r, q);
}

// The roots of v >= 0: the estimate of 22 bits and a step of Heron's iteration,
// which leaves 2^-44 before the rounding.  0 is its own root; infinity and NaN
// give NaN; below 2^-126, where v holds but a few bits, roots come out smaller.
__device__ __forceinline__ float2 root_of(float2 v) {
    float2 r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(fmaxf(v.x, kLeastScale)));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(fmaxf(v.y, kLeastScale)));
    const float2 s = __fmul2_rn(v, r);
    const float2 rest = __ffma2_rn(make_float2(-s.x, -s.y), s, v);
    return __ffma2_rn(rest, __fmul2_rn(r, make_float2(0.5f, 0.5f)), s);
}

__device__ __forceinline__ float reciprocal(float v) {      // to 1 step; v is normal
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float fine_reciprocal(float v) { // Newton's step on it
    const float r = reciprocal(v);
    return fmaf(fmaf(-v, r, 1.f), r, r);
}

__device__ __forceinline__ void from_codes(uint2 w, float scale, float2 (&f)[4]) {
    const uint32_t word[2] = {w.x, w.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(word[j / 2] >> (16 * (j & 1)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
        f[j] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&h)), make_float2(scale, scale));
    }
}

// The scale of a warp's 256 values (magnitudes compare as whole numbers, NaN
// above all).
template <bool SIGNED>
__device__ __forceinline__ float warp_scale(const float2 (&f)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        m = SIGNED ? max(m, max(__float_as_uint(f[j].x) << 1, __float_as_uint(f[j].y) << 1))
                   : max(m, max(__float_as_uint(f[j].x), __float_as_uint(f[j].y)));
    if (SIGNED) m >>= 1;
    return scale_of(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, m)));
}

__device__ __forceinline__ float2 twice(float f) { return make_float2(f, f); }

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
__global__ void __launch_bounds__(kThreads, 4)
    adamw_kernel(const __grid_constant__ TensorTable<N> table, const __grid_constant__ AdamWParams p, int per) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t block = (int64_t)blockIdx.x * kWarps * per + warp;
    if (block >= table.blocks) return;
    const float gs = p.grad_scale ? *p.grad_scale : 1.f;
    if (!(gs > 0.f && gs <= 3.4028234e38f)) return;      // nothing is touched
    const uint64_t t = p.step_dev ? (uint64_t)*p.step_dev : p.step;
    const Step s = step_of(p, t);
    // nor by a step or a rate on the device that the host's numbers may not be
    // (1 - b^0 is no divisor)
    if ((int64_t)t < 1 || !(s.lr >= 0.f && s.lr <= 3.4028234e38f)) return;
    int i = find(table, block);
    for (int k = 0; k < per && block < table.blocks; ++k, block += kWarps) {
        while (i + 1 < table.count && table.t[i + 1].first <= block) ++i;
        const TensorEntry &e = table.t[i];
        const int64_t at = (block - e.first) * kBlock + lane * 8;       // in the tensor
        const int64_t in = e.state + (block - e.first);                 // block of the states
        const int n = e.n - at >= 8 ? 8 : e.n > at ? (int)(e.n - at) : 0;
        const uint32_t pd = e.kind & 3, gd = (e.kind >> 2) & 3;
        float *master = pd != CT_F32 ? p.master + (e.master + block - e.first) * kBlock + lane * 8 : nullptr;
        float2 g[4], w[4], m[4], v[4], root[4];
        uint4 d = {};
        // The next block's lines into L2, one a lane (fp32 moves enough without:
        // 67M elements 271 us, 285 with; with 8-bit states 186, 227 without).
        if (BITS == 8 && k + 1 < per && (block - e.first + kWarps + 1) * kBlock <= e.n) {
            const int64_t next = block - e.first + kWarps, then = in + kWarps;
            const int line = lane & 7;
            const char *from;
            bool more = true;
            if (lane < 8) {
                from = (const char *)e.grad + next * (gd == CT_F32 ? 1024 : 512) + line * 128;
                more = gd == CT_F32 || line < 4;
            } else if (lane < 16) {
                from = (master ? (const char *)(p.master + (e.master + next) * kBlock)
                               : (const char *)e.param + next * 1024) + line * 128;
            } else {
                from = (const char *)(lane < 24 ? p.m : p.v) + then * kBlock + line * 128;
                more = line < 2;
            }
            if (more) asm volatile("prefetch.global.L2 [%0];" ::"l"(from));
        }
        load8(e.grad, gd, at, n, e.kind & kGradVec, g);
        if (master) load8_f32(master, w);
        else load8(e.param, CT_F32, at, n, e.kind & kParamVec, w);
        if (BITS == 32) {
            load8_f32((const float *)p.m + in * kBlock + lane * 8, m);
            load8_f32((const float *)p.v + in * kBlock + lane * 8, v);
        } else {
            const uint2 cm = *reinterpret_cast<const uint2 *>((const uint8_t *)p.m + in * kBlock + lane * 8);
            const uint2 cv = *reinterpret_cast<const uint2 *>((const uint8_t *)p.v + in * kBlock + lane * 8);
            const float sm = p.m_scale[in], sv = p.v_scale[in];
            // the random bits while all that is on its way
            Philox<true> philox(p.rng);
            philox.c2 = (uint32_t)t;
            philox.c3 = (uint32_t)(t >> 32);
            d = philox((uint64_t)(in * (kBlock / 8) + lane));
            from_codes(cm, sm, m);
            from_codes(cv, sv, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(v[j], v[j]);
        }
        if (n < 8) {         // what lies behind the tensor in its last block counts for nothing, and becomes 0
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (2 * j >= n) w[j].x = m[j].x = v[j].x = 0.f;
                if (2 * j + 1 >= n) w[j].y = m[j].y = v[j].y = 0.f;
            }
        }
        const float decay = s.lr * e.decay;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // each operation rounded, as the formulas stand: what 8-bit codes are
            // chosen by is then the same wherever it is computed in fp32
            const float2 a = __fmul2_rn(g[j], twice(gs));
            m[j] = plus(__fmul2_rn(m[j], twice(p.beta1)), __fmul2_rn(a, twice(p.rest1)));
            v[j] = plus(__fmul2_rn(v[j], twice(p.beta2)), __fmul2_rn(__fmul2_rn(a, a), twice(p.rest2)));
            root[j] = root_of(v[j]);
            const float2 q = __ffma2_rn(root[j], twice(s.root_c2), twice(p.eps));
            const float2 u = __fmul2_rn(__fmul2_rn(m[j], make_float2(reciprocal(q.x), reciprocal(q.y))), twice(-s.lr_c1));
            w[j] = __fadd2_rn(w[j], __ffma2_rn(w[j], twice(-decay), u));
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
            const float sm = warp_scale<true>(m), sv = warp_scale<false>(root);
            const float im = fine_reciprocal(sm), iv = fine_reciprocal(sv);
            const uint32_t bits[4] = {d.x, d.y, d.z, d.w};
            uint32_t cm[8], cv[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t r0 = __byte_perm(bits[j], 0, 0x4104), r1 = __byte_perm(bits[j], 0, 0x4324);
                const float2 down = twice(0x1p-120f);
                const float2 x = __fmul2_rn(quotient(m[j], -sm, im), down);
                const float2 y = __fmul2_rn(quotient(root[j], -sv, iv), down);
                cm[2 * j] = code_of(x.x, r0) | (__float_as_uint(x.x) & 0x80000000u);
                cm[2 * j + 1] = code_of(x.y, r1) | (__float_as_uint(x.y) & 0x80000000u);
                // a root above 0 has bits above 1 << 24
                cv[2 * j] = max(code_of(y.x, r0), min(__float_as_uint(root[j].x), 1u << 24));
                cv[2 * j + 1] = max(code_of(y.y, r1), min(__float_as_uint(root[j].y), 1u << 24));
            }
            *reinterpret_cast<uint2 *>((uint8_t *)p.m + in * kBlock + lane * 8) =
                make_uint2(top_bytes(cm[0], cm[1], cm[2], cm[3]), top_bytes(cm[4], cm[5], cm[6], cm[7]));
            *reinterpret_cast<uint2 *>((uint8_t *)p.v + in * kBlock + lane * 8) =
                make_uint2(top_bytes(cv[0], cv[1], cv[2], cv[3]), top_bytes(cv[4], cv[5], cv[6], cv[7]));
            if (lane == 0) {
                p.m_scale[in] = sm;
                p.v_scale[in] = sv;
            }
        }
    }
}

// ---- the gradients' norm ------------------------------------------------------

// The sum of squares to 48 bits and more: a step has billions of them, and its
// scale is to be the same however they are added up.  fp32's squares take 64
// bits.  Those of 16-bit types are exact in fp32; they are added to a sum of two
// floats, each addition with its error (Knuth's sum of two, 1969), and that goes
// to 64 bits after 32 of them (134M bf16 64 us; 78 with a conversion each).
struct Squares {
    double sum = 0.0;

    __device__ __forceinline__ void wide(const float2 (&g)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sum += fma((double)g[j].x, (double)g[j].x, (double)g[j].y * (double)g[j].y);
    }
    // U times eight elements of a type
    template <int U>
    __device__ __forceinline__ void add(const float2 (&g)[U][4], bool narrow) {
        float most = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) most = fmaxf(most, fmaxf(fabsf(g[u][j].x), fabsf(g[u][j].y)));
        // within 2^-50 .. 2^60 no square leaves fp32, nor loses what counts
        if (narrow && most >= 0x1p-50f && most <= 0x1p60f) {
            float2 high = make_float2(0.f, 0.f), low = high;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 q = __fmul2_rn(g[u][j], g[u][j]), s = __fadd2_rn(high, q);
                    const float2 part = minus(s, high), rest = minus(q, part);
                    low = __fadd2_rn(low, __fadd2_rn(minus(high, minus(s, part)), rest));
                    high = s;
                }
            sum += ((double)high.x + (double)high.y) + ((double)low.x + (double)low.y);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) wide(g[u]);
        }
    }
    static __device__ __forceinline__ float2 minus(float2 a, float2 b) { return __fadd2_rn(a, make_float2(-b.x, -b.y)); }
};

// A thread block has a run of blocks; its order and that of the join depend on
// sizes alone.
template <int N>
__global__ void __launch_bounds__(kThreads, 4) norm_kernel(const __grid_constant__ TensorTable<N> table, double *partial) {
    __shared__ double side[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t each = (table.blocks + gridDim.x - 1) / gridDim.x;
    const int64_t first = blockIdx.x * each, last = first + each < table.blocks ? first + each : table.blocks;
    Squares squares;
    if (first + warp < last) {
        int i = find(table, first + warp);
        int64_t block = first + warp;
        while (block < last) {
            while (i + 1 < table.count && table.t[i + 1].first <= block) ++i;
            const TensorEntry &e = table.t[i];
            const int64_t at = (block - e.first) * kBlock + lane * 8;
            const uint32_t gd = (e.kind >> 2) & 3;
            // whole blocks of one tensor, four on their way; the next ones' lines go
            // to L2, one a lane
            constexpr int U = 4, kStep = kWarps * kBlock;
            const int64_t rel = block - e.first;
            if ((rel + (U - 1) * kWarps + 1) * kBlock <= e.n && block + (U - 1) * kWarps < last && (e.kind & kGradVec)) {
                const int lines = gd == CT_F32 ? 8 : 4, ahead = lane / lines;
                if (ahead < U && (rel + (2 * U - 1) * kWarps + 1) * kBlock <= e.n)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(
                        (const char *)e.grad + ((rel + (U + ahead) * kWarps) * lines + lane % lines) * 128));
                float2 g[U][4];
                if (gd == CT_F32) {
#pragma unroll
                    for (int u = 0; u < U; ++u) load8_f32((const float *)e.grad + at + u * kStep, g[u]);
                } else {
                    uint4 raw[U];        // all loaded before the first is looked at
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        raw[u] = *reinterpret_cast<const uint4 *>((const uint16_t *)e.grad + at + u * kStep);
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (gd == CT_F16) unpack(raw[u], g[u], __half());
                        else unpack(raw[u], g[u], __nv_bfloat16());
                }
                squares.add<U>(g, gd != CT_F32);
                block += U * kWarps;
            } else {
                float2 g[1][4];
                load8(e.grad, gd, at, e.n - at >= 8 ? 8 : e.n > at ? (int)(e.n - at) : 0, e.kind & kGradVec, g[0]);
                squares.add<1>(g, gd != CT_F32);
                block += kWarps;
            }
        }
    }
    double sum = squares.sum;
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
    // a norm that fp32 does not hold is none to scale by
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
        // A block a warp.  With 8-bit states, whose warps compute as long as they
        // wait, up to 16 of them one after the other, in whole rounds of resident
        // thread blocks (67M elements: 16 186 us, 8 190, 4 201, 1 242).
        int64_t per = 1;
        if (BITS == 8) {
            const int64_t round = 148 * 4 * kWarps;
            const int64_t waves = ceil_div(table.blocks, round * 16);
            per = ceil_div(table.blocks, round * waves);
        }
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

// f(N): the smallest table that holds `count` tensors, or the largest.
template <typename F>
ct_status by_count(int64_t count, F f) {
    if (count <= kFewTensors) return f(std::integral_constant<int, kFewTensors>());
    if (count <= kSomeTensors) return f(std::integral_constant<int, kSomeTensors>());
    return f(std::integral_constant<int, kManyTensors>());
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
    return by_count(count, [&](auto n) {
        constexpr int N = decltype(n)::value;
        return d->bits == 32 ? adamw_tables<32, N>(count, shapes, params, grads, p, st)
                             : adamw_tables<8, N>(count, shapes, params, grads, p, st);
    });
}

ct_status grad_norm_run(int64_t count, const ct_param *shapes, const void *const *grads, double max_norm, float *norm,
                        float *scale, double *ws, cudaStream_t st) {
    return by_count(count, [&](auto n) {
        return norm_tables<decltype(n)::value>(count, shapes, grads, max_norm, norm, scale, ws, st);
    });
}

}  // namespace ct
