// Root-mean-square norm of rows of C channels, forward and backward:
//
//     h = x + residual,   rstd = (sum_c h^2 / C + eps)^-1/2,   y = h rstd w
//     t = dy w,   dx = rstd (t - h rstd * sum_c (t h rstd) / C) + dsum,   dw = sum_rows dy h rstd
//
// Bound: HBM, with 5 to 12 operations for an element of four tensors.  A row
// therefore stays in the registers of the threads that share it, and every
// tensor is read once.  h is formed in fp32; what goes out as `sum` is rounded,
// y comes from the unrounded values.  Sums are fp32, joined in an order that
// only the sizes set: lanes, warps, then (dw) rows of a block, blocks.
// Measured (GPU time; against the measured copy rate): [8,64x64,1024] bf16 with
// a residual 42 us (0.98), e4m3 [32768,4096] fp16 with a residual 149 (0.96),
// [32768,4096] bf16 without 96 (0.85), backward [16,112x112,512] fp16 with the
// sum's gradient 124 (1.01), rows of 511 bf16 forward 116 (0.71), backward 134
// (0.61).
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "ct_cuda_util.h"
#include "e4m3.cuh"
#include "rms_norm.h"
#include "sm100.cuh"
#include "vec16.cuh"

namespace ct {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kJoinRows = 32;       // partial sums that a block of the join adds side by side

struct RmsParams {
    const void *x, *residual, *weight, *dy, *dsum;
    void *y, *sum, *dx, *dweight;
    float *rstd, *scale;
    const float *rstd_in;
    float *ws;
    int64_t rows, C;
    float eps, inv_c;
    int32_t tpr_log2, wide;                  // wide: the weight is fp32
    int32_t block, block_log2, blocks_c;     // blocks_c: scales per row
    int64_t parts;
};

// E elements of a tensor as they are loaded, a 16-byte vector or one element,
// and as floats.
template <typename T, int E>
using Raw = std::conditional_t<E == 1, T, uint4>;

template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_raw(const T *p) {
    return *reinterpret_cast<const Raw<T, E> *>(p);
}

template <typename T, int E>
__device__ __forceinline__ void of_raw(const Raw<T, E> &r, float (&f)[E]) {
    if constexpr (E == 1) {
        f[0] = to_f<T>(r);
    } else {
        float2 v[E / 2];
        unpack(r, v, T());
#pragma unroll
        for (int j = 0; j < E / 2; ++j) f[2 * j] = v[j].x, f[2 * j + 1] = v[j].y;
    }
}

template <typename T, int E>
__device__ __forceinline__ void load_e(const T *p, float (&f)[E]) {
    of_raw<T, E>(load_raw<T, E>(p), f);
}

template <typename T, int E>
__device__ __forceinline__ void store_e(T *p, const float (&f)[E]) {
    if constexpr (E == 1) {
        *p = from_f<T>(f[0]);
    } else {
        float2 v[E / 2];
#pragma unroll
        for (int j = 0; j < E / 2; ++j) v[j] = make_float2(f[2 * j], f[2 * j + 1]);
        *reinterpret_cast<uint4 *>(p) = pack(v, T());
    }
}

// The weight of E channels from c: 1 where there is none.
template <typename T, int E>
__device__ __forceinline__ void load_weight(const RmsParams &p, int64_t c, float (&f)[E]) {
    if (!p.weight) {
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = 1.f;
    } else if (!p.wide) {
        load_e<T, E>((const T *)p.weight + c, f);
    } else {
        const float *w = (const float *)p.weight + c;
        if constexpr (E == 1) {
            f[0] = *w;
        } else {
#pragma unroll
            for (int j = 0; j < E; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(w + j);
                f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
            }
        }
    }
}

struct Add {
    __device__ static float of(float a, float b) { return a + b; }
};
struct Max {
    __device__ static float of(float a, float b) { return max_nan(a, b); }
};

// One value of all threads of a row, the same in each of them.  `parts`: a
// float for every warp of the block; a block that comes here again uses
// another array in between.
template <typename Op>
__device__ __forceinline__ float across(float v, int tpr_log2, float4 *parts) {
    const int lanes = tpr_log2 < 5 ? 1 << tpr_log2 : 32;
    for (int o = lanes / 2; o > 0; o /= 2) v = Op::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (tpr_log2 <= 5) return v;
    float *const each = reinterpret_cast<float *>(parts);
    const int warp = threadIdx.x >> 5, warps = 1 << (tpr_log2 - 5);
    if ((threadIdx.x & 31) == 0) each[warp] = v;
    __syncthreads();
    const int first = warp & ~(warps - 1);
    if (warps == 2) return Op::of(each[first], each[first + 1]);
    float4 a = parts[first / 4];
    v = Op::of(Op::of(a.x, a.y), Op::of(a.z, a.w));
    for (int w = 1; w < warps / 4; ++w) {
        a = parts[first / 4 + w];
        v = Op::of(v, Op::of(Op::of(a.x, a.y), Op::of(a.z, a.w)));
    }
    return v;
}

// A thread's place in its row: warps take runs of K vectors a lane, so that a
// block of up to 128 channels lies in one warp.  FIXED: a row has whole warps,
// or one vector a thread.
template <int K, bool FIXED>
struct Place {
    int slot;     // row of the block
    int first;    // vector k of this thread is first + k * step
    int step;
    bool lead;    // the row's first thread
    __device__ explicit Place(int tpr_log2) {
        const int t = threadIdx.x & ((1 << tpr_log2) - 1), lanes = FIXED || tpr_log2 > 5 ? 5 : tpr_log2;
        slot = threadIdx.x >> tpr_log2;
        step = 1 << lanes;
        first = FIXED && K == 1 ? t : (t >> lanes << lanes) * K + (t & (step - 1));
        lead = t == 0;
    }
};

// The largest magnitude of the block of channels that each of a thread's
// vectors lies in.  Its lanes are neighbours; where a block has more channels
// than 32 lanes hold, it goes on in the thread's next vectors.
template <int E, int K>
__device__ __forceinline__ void block_max(float (&m)[K], int block) {
    const int lanes = block / E < 32 ? block / E : 32;
    for (int o = lanes / 2; o > 0; o /= 2)
#pragma unroll
        for (int k = 0; k < K; ++k) m[k] = max_nan(m[k], __shfl_xor_sync(0xFFFFFFFFu, m[k], o));
    if constexpr (E == 1 && K >= 2) {
        if (block >= 64)
#pragma unroll
            for (int k = 0; k < K; k += 2) m[k] = m[k + 1] = max_nan(m[k], m[k + 1]);
        if constexpr (K >= 4) {
            if (block >= 128)
#pragma unroll
                for (int k = 0; k < K; k += 4) {
                    const float a = max_nan(m[k], m[k + 2]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) m[k + j] = a;
                }
        }
    }
}

// A thread's K * E elements of a row as pairs (sm_100 adds, multiplies and
// accumulates two floats in one operation): neighbours of a vector, or of E = 1
// two vectors.
template <int E, int K>
struct Elements {
    static constexpr int N = (K * E + 1) / 2;
    float2 v[N];

    // vector k, of a tensor's raw words
    template <typename T>
    __device__ __forceinline__ void set(int k, const Raw<T, E> &r) {
        if constexpr (E == 1) {
            (k & 1 ? v[k / 2].y : v[k / 2].x) = to_f<T>(r);
            if (K == 1) v[0].y = 0.f;
        } else {
            float2 p[E / 2];
            unpack(r, p, T());
#pragma unroll
            for (int j = 0; j < E / 2; ++j) v[k * E / 2 + j] = p[j];
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(int k, T *to) const {
        if constexpr (E == 1) {
            *to = from_f<T>(k & 1 ? v[k / 2].y : v[k / 2].x);
        } else {
            float2 p[E / 2];
#pragma unroll
            for (int j = 0; j < E / 2; ++j) p[j] = v[k * E / 2 + j];
            *reinterpret_cast<uint4 *>(to) = pack(p, T());
        }
    }
    // element j of vector k
    __device__ __forceinline__ float at(int k, int j) const {
        const int i = k * E + j;
        return i & 1 ? v[i / 2].y : v[i / 2].x;
    }
    __device__ __forceinline__ void put(int k, int j, float f) {
        const int i = k * E + j;
        (i & 1 ? v[i / 2].y : v[i / 2].x) = f;
    }
};

// a^-1/2 to half a step more than fp32 holds: the hardware's estimate (22 bits)
// and a step of Newton's iteration.  a = 0 gives infinity, infinity 0.
__device__ __forceinline__ float inverse_root(float a) {
    const float r = rsqrtf(a), e = fmaf(-a * r, r, 1.f);
    return a > 0.f && a <= 3.4028234e38f ? fmaf(0.5f * r, e, r) : r;
}

// What a thread makes of its part of a row, h, once the row's sum is known: y
// or its codes.  `mine`: vectors k with k * step < mine are there; e0: where the
// part starts; w: the weights.
template <typename T, int E, int K, bool Q, bool FULL, typename P>
__device__ __forceinline__ void finish_row(const RmsParams &p, const P &at, int64_t row, int mine, int64_t e0,
                                           Elements<E, K> &h, float sum, const Elements<E, K> &w, float4 *parts) {
    const float rstd = inverse_root(fmaf(sum, p.inv_c, p.eps));
    if (p.rstd && (FULL || mine > 0) && at.lead) p.rstd[row] = rstd;
    const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < h.N; ++i) h.v[i] = __fmul2_rn(__fmul2_rn(h.v[i], r2), w.v[i]);
    if constexpr (!Q) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (FULL || k * at.step < mine) h.store(k, (T *)p.y + e0 + k * at.step * E);
        return;
    }
    float m[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        m[k] = 0.f;
        // what is not there is 0, or 0 * infinity: not looked at
        if (FULL || k * at.step < mine)
#pragma unroll
            for (int j = 0; j < E; ++j) m[k] = max_nan(m[k], fabsf(h.at(k, j)));
    }
    if (p.block == 0) {
#pragma unroll
        for (int k = 1; k < K; ++k) m[0] = max_nan(m[0], m[k]);
        m[0] = scale_of(across<Max>(m[0], p.tpr_log2, parts));
        if ((FULL || mine > 0) && at.lead) p.scale[row] = m[0];
    } else {
        block_max<E, K>(m, p.block);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (at.first + k * at.step) * E;
            m[k] = scale_of(m[k]);
            if ((FULL || k * at.step < mine) && (c & (p.block - 1)) == 0)
                p.scale[row * p.blocks_c + (c >> p.block_log2)] = m[k];
        }
    }
    const float inv0 = 1.f / m[0];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!FULL && k * at.step >= mine) continue;
        const float inv = p.block == 0 || k == 0 ? inv0 : 1.f / m[k];
        uint8_t *q = (uint8_t *)p.y + e0 + k * at.step * E;
        if constexpr (E == 1) {
            *q = (uint8_t)codes2(h.at(k, 0) * inv, 0.f);
        } else {
            const float2 i2 = make_float2(inv, inv);
            uint32_t c[E / 4];
#pragma unroll
            for (int j = 0; j < E / 4; ++j) {
                const float2 a = __fmul2_rn(h.v[k * E / 2 + 2 * j], i2), b = __fmul2_rn(h.v[k * E / 2 + 2 * j + 1], i2);
                c[j] = codes4(a.x, a.y, b.x, b.y);
            }
            if constexpr (E == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(c[0], c[1]);
            else *reinterpret_cast<uint32_t *>(q) = c[0];
        }
    }
}

// The weights of a thread's channels; 0 where it has none.
template <typename T, int E, int K, typename P>
__device__ __forceinline__ void weights_of(const RmsParams &p, const P &at, Elements<E, K> &w) {
#pragma unroll
    for (int i = 0; i < w.N; ++i) w.v[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at.first + k * at.step;
        if (v >= (int)(p.C / E)) continue;
        float f[E];
        load_weight<T, E>(p, (int64_t)v * E, f);
#pragma unroll
        for (int j = 0; j < E; ++j) w.put(k, j, f[j]);
    }
}

template <int E, int K>
__device__ __forceinline__ float squares(const Elements<E, K> &h) {
    float2 both = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < h.N; ++i) both = __ffma2_rn(h.v[i], h.v[i], both);
    return both.x + both.y;
}

// Forward, a row's tensors loaded into registers.  FULL: every thread has K
// vectors of some row, and weights of type W; what is not asked then is most of
// the e4m3 form's work ([32768,4096] fp16 149 us, 178 when it asks).
template <typename T, int E, int K, bool RES, bool Q, typename W>
__global__ void __launch_bounds__(K * E <= kRmsFewElements ? 1024 : kMaxThreads) rms_forward_kernel(const RmsParams p) {
    constexpr bool FULL = !std::is_same_v<W, void>;
    __shared__ float4 parts[2][2][1024 / 128];
    const Place<K, FULL || E == 1> at(p.tpr_log2);
    const int nv = (int)(p.C / E);
    const int64_t rpb = blockDim.x >> p.tpr_log2;
    int turn = 0;
    for (int64_t row0 = blockIdx.x * rpb; row0 < p.rows; row0 += gridDim.x * rpb, turn ^= 1) {
        const int64_t row = row0 + at.slot;
        const int mine = row < p.rows ? nv - at.first : 0;
        const int64_t e0 = row * p.C + (int64_t)at.first * E;
        const T *x = (const T *)p.x + e0, *res = (const T *)p.residual + e0;
        Raw<T, E> rx[K], rr[RES ? K : 1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!FULL) {
                rx[k] = Raw<T, E>();
                if (RES) rr[k] = Raw<T, E>();
            }
            if (FULL || k * at.step < mine) {
                rx[k] = load_raw<T, E>(x + k * at.step * E);
                if (RES) rr[k] = load_raw<T, E>(res + k * at.step * E);
            }
        }
        Elements<E, K> h, w;
#pragma unroll
        for (int k = 0; k < K; ++k) h.template set<T>(k, rx[k]);
        if (RES) {
#pragma unroll
            for (int k = 0; k < K; ++k) w.template set<T>(k, rr[k]);
#pragma unroll
            for (int i = 0; i < h.N; ++i) h.v[i] = __fadd2_rn(h.v[i], w.v[i]);
            if (p.sum)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (FULL || k * at.step < mine) h.store(k, (T *)p.sum + e0 + k * at.step * E);
        }
        const float sum = across<Add>(squares(h), p.tpr_log2, parts[turn][0]);
        if constexpr (!FULL) {
            weights_of<T, E, K>(p, at, w);
        } else if constexpr (std::is_same_v<W, T>) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                w.template set<T>(k, load_raw<T, E>((const T *)p.weight + (at.first + k * at.step) * E));
        } else {
#pragma unroll
            for (int i = 0; i < w.N; i += 2) {      // a vector of 8 elements: two of 4 floats
                const int k = 2 * i / E;
                const float4 f = *reinterpret_cast<const float4 *>((const float *)p.weight +
                                                                   (at.first + k * at.step) * E + 2 * i % E);
                w.v[i] = make_float2(f.x, f.y);
                w.v[i + 1] = make_float2(f.z, f.w);
            }
        }
        finish_row<T, E, K, Q, FULL>(p, at, row, mine, e0, h, sum, w, parts[turn][1]);
    }
}

__device__ __forceinline__ uint32_t shared_address(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes from global to shared memory, past the registers.
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Forward of many rows of whole vectors, without a residual: a block stays for
// row after row, its weights in registers.  The rows come through a ring of S of them in shared
// memory, filled S - 1 ahead by asynchronous copies, so that the bytes in
// flight do not cost registers.  A thread reads what it copied itself: the ring
// needs no barrier.
template <typename T, int E, int K, int S>
__global__ void __launch_bounds__(kMaxThreads) rms_forward_ring_kernel(const RmsParams p) {
    __shared__ float4 parts[2][kMaxThreads / 128];
    extern __shared__ uint4 ring[];                  // [S][K][threads]
    const Place<K, false> at(p.tpr_log2);
    const int nv = (int)(p.C / E);
    const int rpb = blockDim.x >> p.tpr_log2;
    const int64_t stride = (int64_t)gridDim.x * rpb, first = (int64_t)blockIdx.x * rpb;
    const int64_t rounds = first < p.rows ? (p.rows - first + stride - 1) / stride : 0;
    uint4 *const own = ring + threadIdx.x;
    const int line = blockDim.x;
    auto fetch = [&](int64_t i, int s) {
        const int64_t row = first + i * stride + at.slot;
        if (i < rounds && row < p.rows) {
            const T *x = (const T *)p.x + row * p.C + (int64_t)at.first * E;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k * at.step < nv - at.first) copy16(shared_address(own + (s * K + k) * line), x + k * at.step * E);
        }
        copies_end();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i, i);
    Elements<E, K> w;
    weights_of<T, E, K>(p, at, w);
    int s = 0;
    for (int64_t i = 0; i < rounds; ++i) {
        fetch(i + S - 1, s == 0 ? S - 1 : s - 1);
        const int64_t row = first + i * stride + at.slot;
        const int mine = row < p.rows ? nv - at.first : 0;
        copies_wait<S - 1>();
        Elements<E, K> h;
#pragma unroll
        for (int k = 0; k < K; ++k)
            h.template set<T>(k, k * at.step < mine ? own[(s * K + k) * line] : make_uint4(0, 0, 0, 0));
        const float sum = across<Add>(squares(h), p.tpr_log2, parts[i & 1]);
        finish_row<T, E, K, false, false>(p, at, row, mine, row * p.C + (int64_t)at.first * E, h, sum, w, nullptr);
        s = s == S - 1 ? 0 : s + 1;
    }
}

// Rows that no block holds: walked element by element, once for each sum and
// once to write.  A block has a row; only the last walk writes, behind a
// barrier, so that an output may lie on an input.
template <typename T, bool RES, bool Q>
__global__ void __launch_bounds__(kMaxThreads) rms_forward_walk_kernel(const RmsParams p) {
    __shared__ float4 parts[2][kMaxThreads / 128];
    constexpr int kLog2 = 9;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *x = (const T *)p.x + row * p.C, *r = RES ? (const T *)p.residual + row * p.C : nullptr;
        auto h = [&](int64_t c) { return RES ? to_f<T>(x[c]) + to_f<T>(r[c]) : to_f<T>(x[c]); };
        auto y = [&](int64_t c, float v, float rstd) {
            float w[1];
            load_weight<T, 1>(p, c, w);
            return v * rstd * w[0];
        };
        float sum = 0.f;
        for (int64_t c = threadIdx.x; c < p.C; c += kMaxThreads) sum = fmaf(h(c), h(c), sum);
        sum = across<Add>(sum, kLog2, parts[0]);
        const float rstd = inverse_root(fmaf(sum, p.inv_c, p.eps));
        if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
        if (!Q) {
            for (int64_t c = threadIdx.x; c < p.C; c += kMaxThreads) {
                const float v = h(c);
                ((T *)p.y)[row * p.C + c] = from_f<T>(y(c, v, rstd));
                if (RES && p.sum) ((T *)p.sum)[row * p.C + c] = from_f<T>(v);
            }
        } else {
            uint8_t *q = (uint8_t *)p.y + row * p.C;
            if (p.block == 0) {
                float m = 0.f;
                for (int64_t c = threadIdx.x; c < p.C; c += kMaxThreads) m = max_nan(m, fabsf(y(c, h(c), rstd)));
                const float scale = scale_of(across<Max>(m, kLog2, parts[1])), inv = 1.f / scale;
                if (threadIdx.x == 0) p.scale[row] = scale;
                for (int64_t c = threadIdx.x; c < p.C; c += kMaxThreads) {
                    const float v = h(c);
                    q[c] = (uint8_t)codes2(y(c, v, rstd) * inv, 0.f);
                    if (RES && p.sum) ((T *)p.sum)[row * p.C + c] = from_f<T>(v);
                }
            } else {
                // a warp has a block of channels, up to four of them a lane
                const int lane = threadIdx.x & 31, n = p.block / 32;
                for (int64_t b = threadIdx.x >> 5; b < p.blocks_c; b += kMaxThreads / 32) {
                    float v[4], m = 0.f;
                    const int64_t c0 = b * p.block + lane;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t c = c0 + 32 * k;
                        const bool in = k < n && c < p.C;
                        v[k] = in ? h(c) : 0.f;
                        if (in && RES && p.sum) ((T *)p.sum)[row * p.C + c] = from_f<T>(v[k]);
                        v[k] = in ? y(c, v[k], rstd) : 0.f;
                        m = max_nan(m, fabsf(v[k]));
                    }
                    for (int o = 16; o > 0; o /= 2) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                    const float scale = scale_of(m), inv = 1.f / scale;
                    if (lane == 0) p.scale[row * p.blocks_c + b] = scale;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < n && c0 + 32 * k < p.C) q[c0 + 32 * k] = (uint8_t)codes2(v[k] * inv, 0.f);
                }
            }
        }
        __syncthreads();   // before the next row's sums
    }
}

// A block's sums of dw: its rows' one after the other, to its line of the workspace.
template <int E, int K, typename P>
__device__ __forceinline__ void store_dw(const RmsParams &p, const P &at, const float (&dw)[K][E], float *slots) {
    const int rpb = blockDim.x >> p.tpr_log2;
    const int64_t nv = p.C / E;
    float *out = rpb > 1 ? slots + (int64_t)at.slot * p.C : p.ws + (int64_t)blockIdx.x * p.C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at.first + k * at.step;
        if (v < nv)
#pragma unroll
            for (int j = 0; j < E; ++j) out[(int64_t)v * E + j] = dw[k][j];
    }
    if (rpb == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
        float s = slots[c];
        for (int r = 1; r < rpb; ++r) s += slots[(int64_t)r * p.C + c];
        p.ws[(int64_t)blockIdx.x * p.C + c] = s;
    }
}

// Backward of rows of whole vectors.  A thread keeps its columns over all rows
// of its block, their weights and sums of dw in registers; dy, x and dsum come
// through a ring of S rows in shared memory, filled S - 1 rows ahead by
// asynchronous copies, so that the bytes in flight do not cost registers.  A
// thread reads what it copied itself: the ring needs no barrier.  ([16,112x112,
// 512] fp16 124 us; 207 with loads to registers.  16 elements a thread, two
// blocks an SM: 8 elements take 155, three blocks with three rows 129.)
template <typename T, int E, int K, int S, bool DSUM, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 && K * E <= kRmsFewElements ? 2 : 1) rms_backward_kernel(const RmsParams p) {
    constexpr int N = DSUM ? 3 : 2;                  // tensors
    __shared__ float4 parts[2][kMaxThreads / 128];
    extern __shared__ uint4 ring[];                  // [S][N][K][threads]; then dw's slots
    const Place<K, false> at(p.tpr_log2);
    const int nv = (int)(p.C / E);
    const int rpb = blockDim.x >> p.tpr_log2;
    const int64_t stride = (int64_t)gridDim.x * rpb, first = (int64_t)blockIdx.x * rpb;
    const int64_t rounds = first < p.rows ? (p.rows - first + stride - 1) / stride : 0;
    auto slot = [&](int s, int n, int k) { return ring + ((s * N + n) * K + k) * blockDim.x + threadIdx.x; };
    auto fetch = [&](int64_t i) {
        const int64_t row = first + i * stride + at.slot;
        if (i < rounds && row < p.rows) {
            const int s = (int)(i % S);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int v = at.first + k * at.step;
                if (v >= nv) continue;
                const int64_t e = row * p.C + (int64_t)v * E;
                copy16(shared_address(slot(s, 0, k)), (const T *)p.dy + e);
                copy16(shared_address(slot(s, 1, k)), (const T *)p.x + e);
                if (DSUM) copy16(shared_address(slot(s, 2, k)), (const T *)p.dsum + e);
            }
        }
        copies_end();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);
    float w[K][E], dw[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at.first + k * at.step;
        if (v < nv) load_weight<T, E>(p, (int64_t)v * E, w[k]);
#pragma unroll
        for (int j = 0; j < E; ++j) dw[k][j] = 0.f;
    }
    float next = first + at.slot < p.rows ? p.rstd_in[first + at.slot] : 0.f;
    for (int64_t i = 0; i < rounds; ++i) {
        fetch(i + S - 1);
        const int64_t row = first + i * stride + at.slot;
        const bool live = row < p.rows;
        const float rstd = next;
        next = row + stride < p.rows ? p.rstd_in[row + stride] : 0.f;
        copies_wait<S - 1>();
        const int s = (int)(i % S);
        float dot = 0.f;
        uint4 rd[K], rh[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!live || at.first + k * at.step >= nv) continue;
            rd[k] = *slot(s, 0, k);
            rh[k] = *slot(s, 1, k);
            float d[E], h[E];
            of_raw<T, E>(rd[k], d);
            of_raw<T, E>(rh[k], h);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                h[j] *= rstd;
                dw[k][j] = fmaf(d[j], h[j], dw[k][j]);
                dot = fmaf(d[j] * w[k][j], h[j], dot);
            }
        }
        if (!p.dx) continue;
        const float mean = across<Add>(dot, p.tpr_log2, parts[i & 1]) * p.inv_c;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at.first + k * at.step;
            if (!live || v >= nv) continue;
            float d[E], h[E], a[E] = {};
            of_raw<T, E>(rd[k], d);
            of_raw<T, E>(rh[k], h);
            if (DSUM) of_raw<T, E>(*slot(s, 2, k), a);
#pragma unroll
            for (int j = 0; j < E; ++j) a[j] = fmaf(rstd, fmaf(-(h[j] * rstd), mean, d[j] * w[k][j]), a[j]);
            store_e<T, E>((T *)p.dx + row * p.C + (int64_t)v * E, a);
        }
    }
    copies_wait<0>();
    sm100::griddep_launch_dependents();
    if (!p.ws) return;
    if (rpb > 1) __syncthreads();        // dw's slots lie on the ring
    store_dw<E, K>(p, at, dw, (float *)ring);
}

// Backward of other rows, element by element (rows of 511 bf16: weights held
// and a row's addresses made once 134 us, made for each element 192).
template <typename T, int K>
__global__ void __launch_bounds__(kMaxThreads, K <= 8 ? 2 : 1) rms_backward_ones_kernel(const RmsParams p) {
    __shared__ float4 parts[2][kMaxThreads / 128];
    extern __shared__ uint4 ring[];
    const Place<K, true> at(p.tpr_log2);
    const int rpb = blockDim.x >> p.tpr_log2;
    const int own = (int)p.C - at.first;              // element k is there where 32 k < own
    float w[K], dw[K][1];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float f[1] = {0.f};
        if (32 * k < own) load_weight<T, 1>(p, at.first + 32 * k, f);
        w[k] = f[0];
        dw[k][0] = 0.f;
    }
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < p.rows; row0 += (int64_t)gridDim.x * rpb, turn ^= 1) {
        const int64_t row = row0 + at.slot, e0 = row * p.C + at.first;
        const int mine = row < p.rows ? own : 0;
        const T *dy = (const T *)p.dy + e0, *x = (const T *)p.x + e0, *dsum = (const T *)p.dsum + e0;
        const float rstd = mine > 0 ? p.rstd_in[row] : 0.f;
        T rd[K], rh[K], ra[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            rd[k] = rh[k] = ra[k] = from_f<T>(0.f);
            if (32 * k < mine) {
                rd[k] = dy[32 * k];
                rh[k] = x[32 * k];
                if (p.dsum) ra[k] = dsum[32 * k];
            }
        }
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float d = to_f<T>(rd[k]), h = to_f<T>(rh[k]) * rstd;
            dw[k][0] = fmaf(d, h, dw[k][0]);
            dot = 32 * k < mine ? fmaf(d * w[k], h, dot) : dot;
        }
        if (!p.dx) continue;
        const float mean = across<Add>(dot, p.tpr_log2, parts[turn]) * p.inv_c;
        T *dx = (T *)p.dx + e0;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (32 * k < mine)
                dx[32 * k] = from_f<T>(fmaf(rstd, fmaf(-(to_f<T>(rh[k]) * rstd), mean, to_f<T>(rd[k]) * w[k]),
                                            to_f<T>(ra[k])));
    }
    sm100::griddep_launch_dependents();
    if (p.ws) store_dw<1, K>(p, at, dw, (float *)ring);
}

// dx of rows that no block holds.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) rms_backward_walk_kernel(const RmsParams p) {
    __shared__ float4 parts[kMaxThreads / 128];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *x = (const T *)p.x + row * p.C, *dy = (const T *)p.dy + row * p.C;
        const float rstd = p.rstd_in[row];
        auto t = [&](int64_t c) {
            float w[1];
            load_weight<T, 1>(p, c, w);
            return to_f<T>(dy[c]) * w[0];
        };
        float dot = 0.f;
        for (int64_t c = threadIdx.x; c < p.C; c += kMaxThreads) dot = fmaf(t(c), to_f<T>(x[c]) * rstd, dot);
        const float mean = across<Add>(dot, 9, parts) * p.inv_c;
        for (int64_t c = threadIdx.x; c < p.C; c += kMaxThreads) {
            const float d = p.dsum ? to_f<T>(((const T *)p.dsum)[row * p.C + c]) : 0.f;
            ((T *)p.dx)[row * p.C + c] = from_f<T>(fmaf(rstd, fmaf(-(to_f<T>(x[c]) * rstd), mean, t(c)), d));
        }
        __syncthreads();
    }
}

// dw of rows that no block holds: a thread has a column and a part of the rows.
template <typename T>
__global__ void __launch_bounds__(256) rms_columns_kernel(const RmsParams p) {
    const int64_t each = (p.rows + p.parts - 1) / p.parts;
    const int64_t first = blockIdx.y * each, last = first + each < p.rows ? first + each : p.rows;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < p.C; c += (int64_t)gridDim.x * 256) {
        float s = 0.f;
        for (int64_t row = first; row < last; ++row) {
            const int64_t i = row * p.C + c;
            s = fmaf(to_f<T>(((const T *)p.dy)[i]), to_f<T>(((const T *)p.x)[i]) * p.rstd_in[row], s);
        }
        p.ws[blockIdx.y * p.C + c] = s;
    }
}

// The parts of dw, 32 side by side for 32 columns.
template <typename T>
__global__ void __launch_bounds__(32 * kJoinRows) rms_join_kernel(const RmsParams p) {
    __shared__ float side[kJoinRows][33];
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    sm100::griddep_wait();
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < p.C; c0 += (int64_t)gridDim.x * 32) {
        const int64_t c = c0 + lane;
        float s = 0.f;
        if (c < p.C)
            for (int64_t i = r; i < p.parts; i += kJoinRows) s += p.ws[i * p.C + c];
        side[r][lane] = s;
        __syncthreads();
        s = side[lane][r];      // column r of the tile, its parts over the lanes
        for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0 && c0 + r < p.C) {
            if (p.wide) ((float *)p.dweight)[c0 + r] = s;
            else ((T *)p.dweight)[c0 + r] = from_f<T>(s);
        }
        __syncthreads();
    }
}

// ---- host -------------------------------------------------------------------

RmsParams params_of(const RmsArgs &a, const RmsGeom &g) {
    RmsParams p = {};
    p.x = a.x; p.residual = a.residual; p.weight = a.weight; p.dy = a.dy; p.dsum = a.dsum;
    p.y = a.y; p.sum = a.sum; p.dx = a.dx; p.dweight = a.dweight;
    p.rstd = a.rstd; p.scale = a.scale; p.rstd_in = a.rstd_in;
    p.ws = a.dweight ? a.ws : nullptr;
    p.rows = a.rows; p.C = a.C;
    p.eps = a.eps;
    p.inv_c = (float)(1.0 / (double)a.C);
    while ((1 << p.tpr_log2) < g.tpr) ++p.tpr_log2;
    p.wide = a.param_dtype == CT_F32;
    p.block = a.block != 0 && a.block < a.C ? a.block : 0;
    while ((1 << p.block_log2) < p.block) ++p.block_log2;
    p.blocks_c = p.block ? (int32_t)ceil_div(a.C, (int64_t)p.block) : 1;
    return p;
}

template <int V>
struct Int {
    static constexpr int value = V;
};

// f(elements, vectors a thread) with each as a type.
template <typename T, typename F>
void by_geom(const RmsGeom &g, F f) {
    if (g.vec) {
        constexpr int E = kVec<T>;
        if (g.K == 1) f(Int<E>(), Int<1>());
        else if (g.K == 2) f(Int<E>(), Int<2>());
        else if (g.K == 4) f(Int<E>(), Int<4>());
        else f(Int<E>(), Int<8>());
    } else {
        if (g.K == 1) f(Int<1>(), Int<1>());
        else if (g.K == 2) f(Int<1>(), Int<2>());
        else if (g.K == 4) f(Int<1>(), Int<4>());
        else if (g.K == 8) f(Int<1>(), Int<8>());
        else f(Int<1>(), Int<32>());
    }
}

template <typename T, bool RES, bool Q>
ct_status forward_launch(const RmsParams &p, const RmsGeom &g, cudaStream_t st) {
    if (g.K == 0) {
        const int64_t blocks = p.rows < 0x7FFFFFFF ? p.rows : 0x7FFFFFFF;
        rms_forward_walk_kernel<T, RES, Q><<<(unsigned)blocks, kMaxThreads, 0, st>>>(p);
        return launch_status();
    }
    bool fine = true;
    by_geom<T>(g, [&](auto e, auto k) -> void {
        constexpr int E = decltype(e)::value, K = decltype(k)::value;
        if constexpr (E > 1 && K * E <= kRmsFewElements && !RES && !Q) {
            if (g.ring > 0) {
                constexpr int S = rms_forward_stages(K);
                const size_t smem = (size_t)S * K * g.threads * 16;
                auto kernel = rms_forward_ring_kernel<T, E, K, S>;
                static std::atomic<int> ready[64];
                fine = allow_smem(kernel, ready, 224 * 1024);
                if (fine) kernel<<<(unsigned)g.ring, g.threads, smem, st>>>(p);
                return;
            }
        }
        auto direct = [&](auto kernel) { kernel<<<(unsigned)g.blocks, g.threads, 0, st>>>(p); };
        if constexpr (E > 1 && K * E <= kRmsFewElements) {
            const bool full = g.tpr >= 32 && p.C == (int64_t)g.tpr * K * E && p.rows % (g.threads / g.tpr) == 0;
            if (full && p.weight && p.wide) return direct(rms_forward_kernel<T, E, K, RES, Q, float>);
            if (full && p.weight) return direct(rms_forward_kernel<T, E, K, RES, Q, T>);
        }
        direct(rms_forward_kernel<T, E, K, RES, Q, void>);
    });
    return fine ? launch_status() : CT_ERR_DEVICE;
}

template <typename T>
ct_status forward_t(const RmsArgs &a, const RmsGeom &g, cudaStream_t st) {
    const RmsParams p = params_of(a, g);
    if (a.residual) return a.scale ? forward_launch<T, true, true>(p, g, st) : forward_launch<T, true, false>(p, g, st);
    return a.scale ? forward_launch<T, false, true>(p, g, st) : forward_launch<T, false, false>(p, g, st);
}

template <typename T>
ct_status backward_t(const RmsArgs &a, const RmsGeom &g, cudaStream_t st) {
    RmsParams p = params_of(a, g);
    p.parts = 0;
    bool fine = true;
    if (a.rows > 0 && g.K == 0) {
        if (a.dx) {
            const int64_t blocks = p.rows < 0x7FFFFFFF ? p.rows : 0x7FFFFFFF;
            rms_backward_walk_kernel<T><<<(unsigned)blocks, kMaxThreads, 0, st>>>(p);
        }
        if (p.ws) {
            p.parts = rms_parts(p.rows, p.C);
            const int64_t blocks = ceil_div(p.C, (int64_t)256);
            rms_columns_kernel<T><<<dim3((unsigned)blocks, (unsigned)p.parts), 256, 0, st>>>(p);
        }
    } else if (a.rows > 0) {
        p.parts = g.blocks;
        const size_t slots = p.ws && g.threads > g.tpr ? (size_t)(g.threads / g.tpr) * p.C * 4 : 0;
        by_geom<T>(g, [&](auto e, auto k) {
            constexpr int E = decltype(e)::value, K = decltype(k)::value;
            if constexpr (E == 1) {
                rms_backward_ones_kernel<T, K><<<(unsigned)g.blocks, g.threads, slots, st>>>(p);
            } else if constexpr (K * E <= 32) {
                constexpr int S = rms_stages(K);
                const size_t ring = (size_t)S * (p.dsum ? 3 : 2) * K * g.threads * 16;
                const size_t smem = ring > slots ? ring : slots;
                auto go = [&](auto kernel, std::atomic<int> *ready) {
                    if (!allow_smem(kernel, ready, 224 * 1024)) return false;
                    kernel<<<(unsigned)g.blocks, g.threads, smem, st>>>(p);
                    return true;
                };
                static std::atomic<int> ready[4][64];
                if (g.threads == 256)
                    fine = p.dsum ? go(rms_backward_kernel<T, E, K, S, true, 256>, ready[0])
                                  : go(rms_backward_kernel<T, E, K, S, false, 256>, ready[1]);
                else
                    fine = p.dsum ? go(rms_backward_kernel<T, E, K, S, true, 512>, ready[2])
                                  : go(rms_backward_kernel<T, E, K, S, false, 512>, ready[3]);
            }
        });
        if (!fine) return CT_ERR_DEVICE;
    }
    ct_status s = launch_status();
    if (s != CT_OK || !p.dweight) return s;
    cudaLaunchConfig_t cfg = {};
    const int64_t blocks = ceil_div(p.C, (int64_t)32);
    cfg.gridDim = dim3((unsigned)(blocks < 4096 ? blocks : 4096));
    cfg.blockDim = dim3(32 * kJoinRows);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.rows > 0 && g.K != 0 ? 1 : 0;   // behind this call's own kernel only
    if (cudaLaunchKernelEx(&cfg, rms_join_kernel<T>, p) != cudaSuccess) {
        cudaGetLastError();
        return CT_ERR_DEVICE;
    }
    return CT_OK;
}

}  // namespace
}  // namespace ct
