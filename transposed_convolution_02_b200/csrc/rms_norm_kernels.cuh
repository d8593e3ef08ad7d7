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
#pragma once

#include <cuda_runtime.h>

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
    int32_t tpr_log2, wide, block, blocks_c;   // wide: the weight is fp32; blocks_c: scales per row
    int64_t parts;
};

// E elements of a tensor as floats: a 16-byte vector, or one element.
template <typename T, int E>
__device__ __forceinline__ void load_e(const T *p, float (&f)[E]) {
    if constexpr (E == 1) {
        f[0] = to_f<T>(*p);
    } else {
        float2 v[E / 2];
        unpack(*reinterpret_cast<const uint4 *>(p), v, T());
#pragma unroll
        for (int j = 0; j < E / 2; ++j) f[2 * j] = v[j].x, f[2 * j + 1] = v[j].y;
    }
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
__device__ __forceinline__ float across(float v, int tpr_log2, float *parts) {
    const int lanes = tpr_log2 < 5 ? 1 << tpr_log2 : 32;
    for (int o = lanes / 2; o > 0; o /= 2) v = Op::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (tpr_log2 > 5) {
        const int warp = threadIdx.x >> 5, warps = 1 << (tpr_log2 - 5);
        if ((threadIdx.x & 31) == 0) parts[warp] = v;
        __syncthreads();
        const int first = warp & ~(warps - 1);
        v = parts[first];
        for (int w = 1; w < warps; ++w) v = Op::of(v, parts[first + w]);
    }
    return v;
}

// A thread's place in its row: warps take runs of K vectors a lane, so that a
// block of up to 128 channels lies in one warp.
struct Place {
    int64_t slot;    // row of the block
    int first, step; // vector k of this thread: first + k * step
    __device__ Place(int tpr_log2, int K) {
        const int t = threadIdx.x & ((1 << tpr_log2) - 1);
        slot = threadIdx.x >> tpr_log2;
        step = tpr_log2 < 5 ? 1 << tpr_log2 : 32;
        first = (t / step) * step * K + (t & (step - 1));
    }
};

// The largest magnitude of the block of channels that each of a thread's
// vectors lies in.  Its lanes are neighbours; where a block has more channels
// than 32 lanes hold, it goes on in the thread's next vectors (`runs` of them).
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

template <typename T, int E, int K, bool RES, bool Q>
__global__ void __launch_bounds__(kMaxThreads) rms_forward_kernel(const RmsParams p) {
    __shared__ float parts[2][2][kMaxThreads / 32];
    const Place at(p.tpr_log2, K);
    const int64_t nv = p.C / E;
    const int64_t rpb = blockDim.x >> p.tpr_log2;
    int turn = 0;
    for (int64_t row0 = blockIdx.x * rpb; row0 < p.rows; row0 += gridDim.x * rpb, turn ^= 1) {
        const int64_t row = row0 + at.slot;
        const bool live = row < p.rows;
        float h[K][E];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at.first + k * at.step;
            const bool in = live && v < nv;
            if (in) load_e<T, E>((const T *)p.x + row * p.C + (int64_t)v * E, h[k]);
            float r[E] = {};
            if (RES && in) load_e<T, E>((const T *)p.residual + row * p.C + (int64_t)v * E, r);
#pragma unroll
            for (int j = 0; j < E; ++j) h[k][j] = !in ? 0.f : RES ? h[k][j] + r[j] : h[k][j];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at.first + k * at.step;
            if (RES && p.sum && live && v < nv) store_e<T, E>((T *)p.sum + row * p.C + (int64_t)v * E, h[k]);
#pragma unroll
            for (int j = 0; j < E; ++j) sum = fmaf(h[k][j], h[k][j], sum);
        }
        sum = across<Add>(sum, p.tpr_log2, parts[turn][0]);
        const float rstd = 1.f / sqrtf(fmaf(sum, p.inv_c, p.eps));
        if (p.rstd && live && (threadIdx.x & ((1 << p.tpr_log2) - 1)) == 0) p.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at.first + k * at.step;
            float w[E];
            if (v < nv) load_weight<T, E>(p, (int64_t)v * E, w);
#pragma unroll
            for (int j = 0; j < E; ++j) h[k][j] = v < nv ? h[k][j] * rstd * w[j] : 0.f;
            if (!Q && live && v < nv) store_e<T, E>((T *)p.y + row * p.C + (int64_t)v * E, h[k]);
        }
        if constexpr (Q) {
            float m[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                m[k] = 0.f;
#pragma unroll
                for (int j = 0; j < E; ++j) m[k] = max_nan(m[k], fabsf(h[k][j]));
            }
            if (p.block == 0) {
#pragma unroll
                for (int k = 1; k < K; ++k) m[0] = max_nan(m[0], m[k]);
                m[0] = scale_of(across<Max>(m[0], p.tpr_log2, parts[turn][1]));
                if (live && (threadIdx.x & ((1 << p.tpr_log2) - 1)) == 0) p.scale[row] = m[0];
#pragma unroll
                for (int k = 1; k < K; ++k) m[k] = m[0];
            } else {
                block_max<E, K>(m, p.block);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int v = at.first + k * at.step;
                    m[k] = scale_of(m[k]);
                    if (live && v < nv && v * E % p.block == 0) p.scale[row * p.blocks_c + v * E / p.block] = m[k];
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int v = at.first + k * at.step;
                if (!live || v >= nv) continue;
                const float inv = 1.f / m[k];
                uint8_t *q = (uint8_t *)p.y + row * p.C + (int64_t)v * E;
                if constexpr (E == 1) {
                    *q = (uint8_t)codes2(h[k][0] * inv, 0.f);
                } else {
                    uint32_t c[E / 4];
#pragma unroll
                    for (int j = 0; j < E; j += 4)
                        c[j / 4] = codes4(h[k][j] * inv, h[k][j + 1] * inv, h[k][j + 2] * inv, h[k][j + 3] * inv);
                    if constexpr (E == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(c[0], c[1]);
                    else *reinterpret_cast<uint32_t *>(q) = c[0];
                }
            }
        }
    }
}

// Rows that no block holds: walked element by element, once for each sum and
// once to write.  A block has a row; only the last walk writes, behind a
// barrier, so that an output may lie on an input.
template <typename T, bool RES, bool Q>
__global__ void __launch_bounds__(kMaxThreads) rms_forward_walk_kernel(const RmsParams p) {
    __shared__ float parts[2][kMaxThreads / 32];
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
        const float rstd = 1.f / sqrtf(fmaf(sum, p.inv_c, p.eps));
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

// Backward: a thread keeps its columns over all rows of its block, with their
// weights and the sums of dw in registers.
template <typename T, int E, int K>
__global__ void __launch_bounds__(kMaxThreads) rms_backward_kernel(const RmsParams p) {
    __shared__ float parts[2][kMaxThreads / 32];
    extern __shared__ float slots[];
    const Place at(p.tpr_log2, K);
    const int64_t nv = p.C / E;
    const int rpb = blockDim.x >> p.tpr_log2;
    float w[K][E], dw[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at.first + k * at.step;
        if (v < nv) load_weight<T, E>(p, (int64_t)v * E, w[k]);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            dw[k][j] = 0.f;
            if (v >= nv) w[k][j] = 0.f;
        }
    }
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < p.rows; row0 += (int64_t)gridDim.x * rpb, turn ^= 1) {
        const int64_t row = row0 + at.slot;
        const bool live = row < p.rows;
        const float rstd = live ? p.rstd_in[row] : 0.f;
        float h[K][E], t[K][E], dot = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at.first + k * at.step;
            if (live && v < nv) {
                load_e<T, E>((const T *)p.x + row * p.C + (int64_t)v * E, h[k]);
                load_e<T, E>((const T *)p.dy + row * p.C + (int64_t)v * E, t[k]);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) h[k][j] = t[k][j] = 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                h[k][j] *= rstd;
                dw[k][j] = fmaf(t[k][j], h[k][j], dw[k][j]);
                t[k][j] *= w[k][j];
                dot = fmaf(t[k][j], h[k][j], dot);
            }
        if (!p.dx) continue;
        const float mean = across<Add>(dot, p.tpr_log2, parts[turn]) * p.inv_c;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at.first + k * at.step;
            if (!live || v >= nv) continue;
            float d[E] = {};
            if (p.dsum) load_e<T, E>((const T *)p.dsum + row * p.C + (int64_t)v * E, d);
#pragma unroll
            for (int j = 0; j < E; ++j) d[j] = fmaf(rstd, fmaf(-h[k][j], mean, t[k][j]), d[j]);
            store_e<T, E>((T *)p.dx + row * p.C + (int64_t)v * E, d);
        }
    }
    sm100::griddep_launch_dependents();
    if (!p.ws) return;
    // the block's rows, one after the other; then its line of the workspace
    float *out = rpb > 1 ? slots + at.slot * p.C : p.ws + (int64_t)blockIdx.x * p.C;
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

// dx of rows that no block holds.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) rms_backward_walk_kernel(const RmsParams p) {
    __shared__ float parts[kMaxThreads / 32];
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
    p.blocks_c = p.block ? (int32_t)ceil_div(a.C, (int64_t)p.block) : 1;
    return p;
}

template <int V>
struct Int {
    static constexpr int value = V;
};

// f(elements, vectors a thread) with each as a type.
template <typename T, bool BACK, typename F>
void by_geom(const RmsGeom &g, F f) {
    if (g.vec) {
        constexpr int E = kVec<T>;
        if (g.K == 1) f(Int<E>(), Int<1>());
        else if (g.K == 2) f(Int<E>(), Int<2>());
        else if (g.K == 4) f(Int<E>(), Int<4>());
        else if constexpr (!BACK || E == 4) f(Int<E>(), Int<8>());
    } else {
        if (g.K == 2) f(Int<1>(), Int<2>());
        else if (g.K == 4) f(Int<1>(), Int<4>());
        else if (g.K == 8) f(Int<1>(), Int<8>());
        else f(Int<1>(), Int<32>());
    }
}

template <typename T, bool RES, bool Q>
void forward_launch(const RmsParams &p, const RmsGeom &g, cudaStream_t st) {
    if (g.K == 0) {
        const int64_t blocks = p.rows < 0x7FFFFFFF ? p.rows : 0x7FFFFFFF;
        rms_forward_walk_kernel<T, RES, Q><<<(unsigned)blocks, kMaxThreads, 0, st>>>(p);
        return;
    }
    by_geom<T, false>(g, [&](auto e, auto k) {
        rms_forward_kernel<T, decltype(e)::value, decltype(k)::value, RES, Q>
            <<<(unsigned)g.blocks, g.threads, 0, st>>>(p);
    });
}

template <typename T>
ct_status forward_t(const RmsArgs &a, const RmsGeom &g, cudaStream_t st) {
    const RmsParams p = params_of(a, g);
    if (a.residual) {
        if (a.scale) forward_launch<T, true, true>(p, g, st);
        else forward_launch<T, true, false>(p, g, st);
    } else {
        if (a.scale) forward_launch<T, false, true>(p, g, st);
        else forward_launch<T, false, false>(p, g, st);
    }
    return launch_status();
}

template <typename T>
ct_status backward_t(const RmsArgs &a, const RmsGeom &g, cudaStream_t st) {
    RmsParams p = params_of(a, g);
    p.parts = 0;
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
        const int rpb = g.threads / g.tpr;
        const size_t smem = p.ws && rpb > 1 ? (size_t)rpb * p.C * 4 : 0;    // at most threads * K * E * 4 = 32 KB
        by_geom<T, true>(g, [&](auto e, auto k) {
            rms_backward_kernel<T, decltype(e)::value, decltype(k)::value>
                <<<(unsigned)g.blocks, g.threads, smem, st>>>(p);
        });
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
