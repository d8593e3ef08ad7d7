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
// a residual 42 us (0.98), e4m3 [32768,4096] fp16 with a residual 139 (1.04),
// [32768,4096] bf16 without 85 (0.96), backward [16,112x112,512] fp16 with the
// sum's gradient 124 (1.01), rows of 511 bf16 forward 100 (0.82), backward 132
// (0.62).
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
    int32_t lanes_log2, warps, rpb;          // of a row: lanes (32 in `warps` warps); rows of a block
    int32_t per_warp, room_log2;             // 65536 / warps, rounded up; floats in shared memory for a row's warps
    int32_t wide;                            // the weight is fp32
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

// A thread's place in its row: warps take runs of K vectors a lane, so that a
// block of up to 128 channels lies in one warp.  FIXED: a row has whole warps,
// or one vector a thread.  WHOLE: it has whole warps (of single elements: more
// than one a thread; rows of 67 fp32 elements 67 % of the floor, 58 when asked).
template <int K, bool FIXED, bool WHOLE = false>
struct Place {
    int slot, warp;    // row of the block; warp of the row
    int first;         // vector k of this thread is first + k * step
    int step;
    bool lead;         // the row's first thread
    __device__ explicit Place(const RmsParams &p) {
        if (WHOLE || p.lanes_log2 == 5) {
            warp = threadIdx.x >> 5;
            slot = warp * p.per_warp >> 16;
            warp -= slot * p.warps;
            first = warp * 32 * K + (threadIdx.x & 31);
            step = 32;
        } else {
            warp = 0;
            slot = threadIdx.x >> p.lanes_log2;
            first = threadIdx.x & ((1 << p.lanes_log2) - 1);
            step = FIXED ? 32 : 1 << p.lanes_log2;
        }
        lead = first == 0;
    }
    static constexpr bool whole = WHOLE;
};

// Room for one value of each warp, a row's from a power of two on: what is left
// between them is 0, for good.
__device__ __forceinline__ void clear(const RmsParams &p, float4 *parts, int n) {
    if (p.warps != 1 << p.room_log2) {
        for (int i = threadIdx.x; i < n; i += blockDim.x) parts[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();
    }
}

// One value of all threads of a row, the same in each of them.  A block that
// comes here again uses another `parts` in between.
template <typename Op, typename P>
__device__ __forceinline__ float across(float v, const RmsParams &p, const P &at, float4 *parts) {
    if (P::whole || p.lanes_log2 == 5) {
#pragma unroll
        for (int o = 16; o > 0; o /= 2) v = Op::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    } else {
        for (int o = (1 << p.lanes_log2) / 2; o > 0; o /= 2) v = Op::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    }
    if (p.warps == 1) return v;
    float *const each = reinterpret_cast<float *>(parts) + (at.slot << p.room_log2);
    if ((threadIdx.x & 31) == 0) each[at.warp] = v;
    __syncthreads();
    if (p.warps == 2) return Op::of(each[0], each[1]);
    const float4 *const all = reinterpret_cast<const float4 *>(each);
    float4 a = all[0];
    v = Op::of(Op::of(a.x, a.y), Op::of(a.z, a.w));
    for (int w = 1; w < 1 << p.room_log2 >> 2; ++w) {
        a = all[w];
        v = Op::of(v, Op::of(Op::of(a.x, a.y), Op::of(a.z, a.w)));
    }
    return v;
}

// A row that starts inside a vector, at its element s, as rows of no whole
// number of vectors do.  All rows of a slot start alike: the host steps by as
// many rows as bring the start back.
template <int E, bool SHIFT>
struct Cut {
    int s = 0, nv, tail = E;
    __device__ Cut(const RmsParams &p, int64_t row) {
        if (SHIFT) {
            s = (int)(row * p.C & (E - 1));
            nv = (int)(s + p.C + E - 1) / E;
            tail = (int)(s + p.C) - (nv - 1) * E;
        } else {
            nv = (int)(p.C / E);
        }
    }
    // which elements of vector v are the row's
    __device__ __forceinline__ uint32_t bits(int v) const {
        uint32_t b = (1u << E) - 1;
        if (SHIFT && v == 0) b &= ~((1u << s) - 1);
        if (SHIFT && v == nv - 1) b &= (1u << tail) - 1;
        return b;
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
    // elements of vector k that are not in `bits` become 0
    __device__ __forceinline__ void keep(int k, uint32_t bits) {
        if (bits == (1u << E) - 1) return;
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (!((bits >> j) & 1)) put(k, j, 0.f);
    }
    template <typename T>
    __device__ __forceinline__ void store(int k, T *to, uint32_t bits) const {
        if (bits == (1u << E) - 1) return store(k, to);
#pragma unroll
        for (int j = 0; j < E; ++j)
            if ((bits >> j) & 1) to[j] = from_f<T>(at(k, j));
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

// The scale of a block of codes: NaN where the largest magnitude is infinite too
// (0 times it is NaN; others this leaves as they are), as a finite h has where
// the weight's product passes fp32.
__device__ __forceinline__ float scale_of_codes(float amax) { return scale_of(fmaf(amax, 0.f, amax)); }

// What a thread makes of its part of a row, h, once the row's sum is known: y
// or its codes.  `mine`: vectors k with k * step < mine are there; e0: where the
// part starts; w: the weights.
template <typename T, int E, int K, bool Q, bool FULL, bool SHIFT, typename P>
__device__ __forceinline__ void finish_row(const RmsParams &p, const P &at, const Cut<E, SHIFT> &cut, int64_t row,
                                           int mine, int64_t e0, Elements<E, K> &h, float sum,
                                           const Elements<E, K> &w, float4 *parts) {
    const float rstd = inverse_root(fmaf(sum, p.inv_c, p.eps));
    if (p.rstd && (FULL || mine > 0) && at.lead) p.rstd[row] = rstd;
    const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < h.N; ++i) h.v[i] = __fmul2_rn(__fmul2_rn(h.v[i], r2), w.v[i]);
    if constexpr (!Q) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (FULL || k * at.step < mine) {
                if (SHIFT) h.store(k, (T *)p.y + e0 + k * at.step * E, cut.bits(at.first + k * at.step));
                else h.store(k, (T *)p.y + e0 + k * at.step * E);
            }
        return;
    }
    float m[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        m[k] = 0.f;
        // what is not there is 0, or 0 * infinity: not looked at
        if (FULL || k * at.step < mine) {
            if constexpr (SHIFT) {
                const uint32_t bits = cut.bits(at.first + k * at.step);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if ((bits >> j) & 1) m[k] = max_nan(m[k], fabsf(h.at(k, j)));
            } else if constexpr (E == 1) {
                m[k] = fabsf(h.at(k, 0));
            } else {
#pragma unroll
                for (int j = 0; j < E; j += 2) m[k] = max_abs_nan(m[k], h.at(k, j), h.at(k, j + 1));
            }
        }
    }
    if (SHIFT || p.block == 0) {
#pragma unroll
        for (int k = 1; k < K; ++k) m[0] = max_nan(m[0], m[k]);
        m[0] = scale_of_codes(across<Max>(m[0], p, at, parts));
        if ((FULL || mine > 0) && at.lead) p.scale[row] = m[0];
    } else {
        block_max<E, K>(m, p.block);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (at.first + k * at.step) * E;
            m[k] = scale_of_codes(m[k]);
            if ((FULL || k * at.step < mine) && (c & (p.block - 1)) == 0)
                p.scale[row * p.blocks_c + (c >> p.block_log2)] = m[k];
        }
    }
    const float inv0 = 1.f / m[0];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!FULL && k * at.step >= mine) continue;
        const float inv = SHIFT || p.block == 0 || k == 0 ? inv0 : 1.f / m[k];
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
            const uint32_t bits = cut.bits(at.first + k * at.step);
            if (SHIFT && bits != (1u << E) - 1) {
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if ((bits >> j) & 1) q[j] = (uint8_t)(c[j / 4] >> (8 * (j & 3)));
            } else if constexpr (E == 8) {
                *reinterpret_cast<uint2 *>(q) = make_uint2(c[0], c[1]);
            } else {
                *reinterpret_cast<uint32_t *>(q) = c[0];
            }
        }
    }
}

// The weights of a thread's channels; 0 where it has none.
template <typename T, int E, int K, bool SHIFT, typename P>
__device__ __forceinline__ void weights_of(const RmsParams &p, const P &at, const Cut<E, SHIFT> &cut,
                                           Elements<E, K> &w) {
#pragma unroll
    for (int i = 0; i < w.N; ++i) w.v[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at.first + k * at.step;
        if (v >= cut.nv) continue;
        if constexpr (SHIFT) {
            const uint32_t bits = cut.bits(v);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                float f[1] = {0.f};
                if ((bits >> j) & 1) load_weight<T, 1>(p, (int64_t)v * E + j - cut.s, f);
                w.put(k, j, f[0]);
            }
        } else {
            float f[E];
            load_weight<T, E>(p, (int64_t)v * E, f);
#pragma unroll
            for (int j = 0; j < E; ++j) w.put(k, j, f[j]);
        }
    }
}

template <int E, int K>
__device__ __forceinline__ float squares(const Elements<E, K> &h) {
    float2 both = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < h.N; ++i) both = __ffma2_rn(h.v[i], h.v[i], both);
    return both.x + both.y;
}

// Registers of a thread of rms_forward_kernel.  The fewer, the more blocks read
// while others sum up.  bf16 with a residual, of the floor: e4m3 of 1024 channels
// 94 % with 40, 91 with 48, 84 with 64; 8192 channels, without codes, 95 with 40
// (three blocks an SM), 86 with 48 (two); 1024 channels 97 with 40, 98 with 48.
// 256 channels, 8 elements a thread, as e4m3: 90 with 32, 83 with 40.  Without a
// residual 1024 channels 87 with 32, 85 with 40; as e4m3, 62 with 40, 52 with 32
// (spilled).
constexpr int rms_forward_registers(int E, int K, bool res, bool codes, bool full, bool wide) {
    if (E == 1) return K <= 4 ? 32 : K == 8 ? (codes ? 48 : 40) : K == 16 ? 64 : 128;
    if (K * E <= 8) return 32;
    if (full && E == 8 && K == 2 && !res && !codes && !wide) return 32;
    if (K * E <= kRmsFewElements) return full && (E == 8 ? codes || wide : codes && !res) ? 40 : 48;
    return K * E <= 24 ? (full ? 56 : 64) : 128;
}

// Forward, a row's tensors loaded into registers.  FULL: every thread has K
// vectors of one row, of at most 2^31, and weights of type W; what is not asked then is most of
// the e4m3 form's work ([32768,4096] fp16, each with 64 registers: 149 us, 178
// when it asks).  WIDE: more than 256 threads.
template <typename T, int E, int K, bool RES, bool Q, typename W, bool WIDE = false>
__global__ void __maxnreg__(rms_forward_registers(E, K, RES, Q, !std::is_same_v<W, void>, WIDE))
    rms_forward_kernel(const RmsParams p) {
    constexpr bool FULL = !std::is_same_v<W, void>;
    __shared__ float4 parts[4][1024 / 128];
    const Place<K, FULL || E == 1, FULL || (E == 1 && K > 1)> at(p);
    const Cut<E, false> cut(p, 0);
    clear(p, parts[0], sizeof(parts) / 16);
    // FULL: the grid has a slot for every row, and no loop is needed; where the
    // codes' kernel has 16 elements in 40 registers, its addresses crowd them
    // ([32768,4096] fp16 with a residual 141 us, 139 with the loop; 256 bf16
    // channels without a residual 60 % of the floor, 50 with it).
    constexpr bool ONCE = FULL && !(Q && K * E == kRmsFewElements && (RES || E == 4));
    const int64_t rpb = p.rpb, last = ONCE ? 1 : p.rows;
    int turn = 0;
    for (int64_t row0 = ONCE ? 0 : blockIdx.x * rpb; row0 < last; row0 += ONCE ? 1 : gridDim.x * rpb, turn ^= 1) {
        const int64_t row = ONCE ? (int64_t)(blockIdx.x * (uint32_t)p.rpb + at.slot) : row0 + at.slot;
        const int mine = row < p.rows ? cut.nv - at.first : 0;
        const int64_t e0 = (ONCE ? (int64_t)((uint64_t)(uint32_t)row * (uint32_t)p.C) : row * p.C) +
                           (int64_t)at.first * E;
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
        const float sum = across<Add>(squares(h), p, at, parts[2 * turn]);
        if constexpr (!FULL) {
            weights_of<T, E, K>(p, at, cut, w);
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
        finish_row<T, E, K, Q, FULL>(p, at, cut, row, mine, e0, h, sum, w, parts[2 * turn + 1]);
    }
}

__device__ __forceinline__ uint32_t shared_address(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes from global to shared memory, past the registers; of the last vector
// of a tensor what there is, and zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_some(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Forward of many rows: a block stays for row after row, its weights in
// registers.  The rows come through a ring of S of them in shared memory, filled
// S - 1 ahead by asynchronous copies, so that the bytes in flight do not cost
// registers.  A thread reads what it copied itself: the ring needs no barrier.
template <typename T, int K, int S, bool RES, bool Q, bool SHIFT>
__global__ void __launch_bounds__(kMaxThreads) rms_forward_ring_kernel(const RmsParams p) {
    constexpr int E = kVec<T>, N = RES ? 2 : 1;      // tensors
    __shared__ float4 parts[4][kMaxThreads / 128];
    extern __shared__ uint4 ring[];                  // [S][N][K][threads]
    const Place<K, false> at(p);
    clear(p, parts[0], sizeof(parts) / 16);
    const int64_t stride = (int64_t)gridDim.x * p.rpb, first = (int64_t)blockIdx.x * p.rpb;
    const int64_t rounds = first < p.rows ? (p.rows - first + stride - 1) / stride : 0;
    const Cut<E, SHIFT> cut(p, first + at.slot);
    const int64_t all = p.rows * p.C;
    uint4 *const own = ring + threadIdx.x;
    const int line = blockDim.x;
    auto fetch = [&](int64_t i, int s) {
        const int64_t row = first + i * stride + at.slot;
        if (i < rounds && row < p.rows) {
            const int64_t e0 = row * p.C - cut.s + (int64_t)at.first * E;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (k * at.step >= cut.nv - at.first) continue;
                const int64_t e = e0 + k * at.step * E;
                const uint32_t to = shared_address(own + (s * N * K + k) * line);
                const int64_t rest = (all - e) * (int)sizeof(T);
                if (SHIFT && rest < 16) {
                    copy_some(to, (const T *)p.x + e, (int)rest);
                    if (RES) copy_some(to + K * line * 16, (const T *)p.residual + e, (int)rest);
                } else {
                    copy16(to, (const T *)p.x + e);
                    if (RES) copy16(to + K * line * 16, (const T *)p.residual + e);
                }
            }
        }
        copies_end();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i, i);
    Elements<E, K> w;
    weights_of<T, E, K>(p, at, cut, w);
    int s = 0;
    for (int64_t i = 0; i < rounds; ++i) {
        fetch(i + S - 1, s == 0 ? S - 1 : s - 1);
        const int64_t row = first + i * stride + at.slot;
        const int mine = row < p.rows ? cut.nv - at.first : 0;
        const int64_t e0 = row * p.C - cut.s + (int64_t)at.first * E;
        copies_wait<S - 1>();
        Elements<E, K> h;
#pragma unroll
        for (int k = 0; k < K; ++k)
            h.template set<T>(k, k * at.step < mine ? own[(s * N * K + k) * line] : make_uint4(0, 0, 0, 0));
        if (RES) {
            Elements<E, K> r;
#pragma unroll
            for (int k = 0; k < K; ++k)
                r.template set<T>(k, k * at.step < mine ? own[((s * N + 1) * K + k) * line] : make_uint4(0, 0, 0, 0));
#pragma unroll
            for (int j = 0; j < h.N; ++j) h.v[j] = __fadd2_rn(h.v[j], r.v[j]);
        }
        if (SHIFT)
#pragma unroll
            for (int k = 0; k < K; ++k) h.keep(k, cut.bits(at.first + k * at.step));
        if (RES && p.sum)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k * at.step < mine)
                    h.store(k, (T *)p.sum + e0 + k * at.step * E, cut.bits(at.first + k * at.step));
        const float sum = across<Add>(squares(h), p, at, parts[2 * (i & 1)]);
        finish_row<T, E, K, Q, false>(p, at, cut, row, mine, e0, h, sum, w, parts[2 * (i & 1) + 1]);
        s = s == S - 1 ? 0 : s + 1;
    }
}

// Rows that no block holds: walked element by element, once for each sum and
// once to write.  A block has a row; only the last walk writes, behind a
// barrier, so that an output may lie on an input.  A thread's sum is one of 64
// bits here: terms that are alike round alike, and 32768 of them (2^24 channels
// of 1.1) were 4e-4 off in fp32.
template <typename T, bool RES, bool Q>
__global__ void __launch_bounds__(kMaxThreads) rms_forward_walk_kernel(const RmsParams p) {
    __shared__ float4 parts[2][kMaxThreads / 128];
    const Place<1, true> at(p);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *x = (const T *)p.x + row * p.C, *r = RES ? (const T *)p.residual + row * p.C : nullptr;
        auto h = [&](int64_t c) { return RES ? to_f<T>(x[c]) + to_f<T>(r[c]) : to_f<T>(x[c]); };
        auto y = [&](int64_t c, float v, float rstd) {
            float w[1];
            load_weight<T, 1>(p, c, w);
            return v * rstd * w[0];
        };
        double squares = 0.0;
        for (int64_t c = threadIdx.x; c < p.C; c += kMaxThreads) squares = fma((double)h(c), (double)h(c), squares);
        const float sum = across<Add>((float)squares, p, at, parts[0]);
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
                const float scale = scale_of_codes(across<Max>(m, p, at, parts[1])), inv = 1.f / scale;
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
                    const float scale = scale_of_codes(m), inv = 1.f / scale;
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
    float *out = p.rpb > 1 ? slots + (int64_t)at.slot * p.C : p.ws + (int64_t)blockIdx.x * p.C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at.first + k * at.step;
        if (v < (int)(p.C / E))
#pragma unroll
            for (int j = 0; j < E; ++j) out[(int64_t)v * E + j] = dw[k][j];
    }
    if (p.rpb == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
        float s = slots[c];
        for (int r = 1; r < p.rpb; ++r) s += slots[(int64_t)r * p.C + c];
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
template <typename T, int K, int S, bool DSUM, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 && K * kVec<T> <= kRmsFewElements ? 2 : 1)
    rms_backward_kernel(const RmsParams p) {
    constexpr int E = kVec<T>, N = DSUM ? 3 : 2;     // tensors
    __shared__ float4 parts[2][kMaxThreads / 128];
    extern __shared__ uint4 ring[];                  // [S][N][K][threads]; then dw's slots
    const Place<K, false> at(p);
    clear(p, parts[0], sizeof(parts) / 16);
    const int rpb = p.rpb;
    const int64_t stride = (int64_t)gridDim.x * rpb, first = (int64_t)blockIdx.x * rpb;
    const int64_t rounds = first < p.rows ? (p.rows - first + stride - 1) / stride : 0;
    const int nv = (int)(p.C / E);
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
        const float mean = across<Add>(dot, p, at, parts[i & 1]) * p.inv_c;
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
    const Place<K, true, (K > 1)> at(p);
    clear(p, parts[0], sizeof(parts) / 16);
    const int rpb = p.rpb;
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
        const float mean = across<Add>(dot, p, at, parts[turn]) * p.inv_c;
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
    const Place<1, true> at(p);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *x = (const T *)p.x + row * p.C, *dy = (const T *)p.dy + row * p.C;
        const float rstd = p.rstd_in[row];
        auto t = [&](int64_t c) {
            float w[1];
            load_weight<T, 1>(p, c, w);
            return to_f<T>(dy[c]) * w[0];
        };
        double dot = 0.0;
        for (int64_t c = threadIdx.x; c < p.C; c += kMaxThreads)
            dot += (double)(t(c) * (to_f<T>(x[c]) * rstd));
        const float mean = across<Add>((float)dot, p, at, parts) * p.inv_c;
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
        float s = 0.f;       // 128 rows by themselves, for the same reason
        for (int64_t row = first; row < last; row += 128) {
            const int n = last - row < 128 ? (int)(last - row) : 128;
            int64_t i = row * p.C + c;
            float part = 0.f;
            for (int k = 0; k < n; ++k, i += p.C)
                part = fmaf(to_f<T>(((const T *)p.dy)[i]), to_f<T>(((const T *)p.x)[i]) * p.rstd_in[row + k], part);
            s += part;
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
    p.lanes_log2 = g.lanes_log2;
    p.warps = g.warps;
    p.per_warp = (65536 + g.warps - 1) / g.warps;
    while (1 << p.room_log2 < g.warps) ++p.room_log2;
    p.rpb = g.rpb;
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

// f(vectors a thread) with the number as a type.
template <typename F>
void by_k(int K, F f) {
    if (K == 1) f(Int<1>());
    else if (K == 2) f(Int<2>());
    else if (K == 3) f(Int<3>());
    else if (K == 4) f(Int<4>());
    else if (K == 8) f(Int<8>());
    else if (K == 16) f(Int<16>());
    else f(Int<32>());
}

template <typename T, bool RES, bool Q>
ct_status forward_launch(const RmsParams &p, const RmsGeom &g, cudaStream_t st) {
    if (g.K == 0) {
        const int64_t blocks = p.rows < 0x7FFFFFFF ? p.rows : 0x7FFFFFFF;
        rms_forward_walk_kernel<T, RES, Q><<<(unsigned)blocks, kMaxThreads, 0, st>>>(p);
        return launch_status();
    }
    bool fine = true;
    auto direct = [&](auto kernel) { kernel<<<(unsigned)g.blocks, g.threads, 0, st>>>(p); };
    by_k(g.K, [&](auto k) -> void {
        constexpr int K = decltype(k)::value, E = kVec<T>;
        if (!g.vec) {
            if constexpr (K != 3 && K <= 16) direct(rms_forward_kernel<T, 1, K, RES, Q, void>);
            return;
        }
        if constexpr (K <= 4) {
            if (g.ring > 0) {
                constexpr int S = rms_forward_stages(K);
                const size_t smem = (size_t)S * (RES ? 2 : 1) * K * g.threads * 16;
                auto stay = [&](auto kernel, std::atomic<int> *ready) {
                    fine = allow_smem(kernel, ready, 224 * 1024);
                    if (fine) kernel<<<(unsigned)g.ring, g.threads, smem, st>>>(p);
                };
                static std::atomic<int> ready[2][64];
                if (g.shift) {
                    if constexpr (E == 8) stay(rms_forward_ring_kernel<T, K, S, RES, Q, true>, ready[0]);
                } else if constexpr (!RES && !Q && (E == 8 || K == 1 || K == 4)) {
                    stay(rms_forward_ring_kernel<T, K, S, RES, Q, false>, ready[1]);
                }
                return;
            }
            if constexpr (K * E <= 24) {
                const bool full = g.lanes_log2 == 5 && p.C == (int64_t)32 * g.warps * K * E && p.rows % g.rpb == 0 &&
                                  p.rows <= 0x7FFFFFFF;
                constexpr bool WIDE = E == 8 && K == 2 && !Q;
                if (full && p.weight) {
                    if (WIDE && g.threads > 256)
                        return p.wide ? direct(rms_forward_kernel<T, E, K, RES, Q, float, WIDE>)
                                      : direct(rms_forward_kernel<T, E, K, RES, Q, T, WIDE>);
                    return p.wide ? direct(rms_forward_kernel<T, E, K, RES, Q, float>)
                                  : direct(rms_forward_kernel<T, E, K, RES, Q, T>);
                }
            }
        }
        // four vectors of 16-bit elements: rows of the ring that are too few for it
        if constexpr (E == 8 ? K <= 3 || K == 8 || (K == 4 && !RES && !Q) : K <= 4)
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
        const size_t slots = p.ws && g.rpb > 1 ? (size_t)g.rpb * p.C * 4 : 0;
        by_k(g.K, [&](auto k) -> void {
            constexpr int K = decltype(k)::value, E = kVec<T>;
            if (!g.vec) {
                if constexpr (K != 3)
                    rms_backward_ones_kernel<T, K><<<(unsigned)g.blocks, g.threads, slots, st>>>(p);
            } else if constexpr (K * E <= 32 && (E == 4 || K != 3)) {
                constexpr int S = rms_stages(K);
                const size_t ring = (size_t)S * (p.dsum ? 3 : 2) * K * g.threads * 16;
                const size_t smem = ring > slots ? ring : slots;
                auto go = [&](auto kernel, std::atomic<int> *ready) {
                    fine = allow_smem(kernel, ready, 224 * 1024);
                    if (fine) kernel<<<(unsigned)g.blocks, g.threads, smem, st>>>(p);
                };
                static std::atomic<int> ready[4][64];
                if (g.threads <= 256) {
                    if (p.dsum) go(rms_backward_kernel<T, K, S, true, 256>, ready[0]);
                    else go(rms_backward_kernel<T, K, S, false, 256>, ready[1]);
                } else {
                    if (p.dsum) go(rms_backward_kernel<T, K, S, true, 512>, ready[2]);
                    else go(rms_backward_kernel<T, K, S, false, 512>, ready[3]);
                }
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
