// Channels-last group norm with its activation and dropout, forward and
// backward.
//
// Per image n and group g (C/G channels, all S pixels, M = S*C/G values):
//   mean = sum x / M,  var = sum (x - mean)^2 / M,  rstd = (var + eps)^-1/2,
//   h = (x - mean) rstd,  a = h w + b,  y = drop(act(a)).
// With da = drop(dy) act'(a) and dh = da w:
//   dw = sum da h,  db = sum da  (over images and pixels),
//   dx = rstd (dh - mean(dh) - h mean(dh h))  (means over the group).
//
// Bound: HBM.  Forward must read x and write y, backward read x and dy and
// write dx.
//
// Statistics: a thread sums x - k and (x - k)^2 of its few values per
// channel, k being the first of them, then everything is merged as (count,
// mean, M2) with M2 the sum of squared distances from the mean.  As k is one
// of the n values summed, sum (x - k)^2 <= n M2, so the subtraction that
// gives M2 loses at most a factor of the thread's n, however far the mean is
// from 0.
#include <string.h>

#include "group_norm.h"
#include "vec8.cuh"

namespace ct {

namespace {

constexpr int kThreads = 256;

struct Params {      // kernel arguments besides the geometry
    const void *x, *dy, *weight, *bias;
    void *y, *dx, *dweight, *dbias;
    float *mean, *rstd;
    float *part, *sums, *coef;
    float eps;
    int param_dtype;
    bool vec;
    RngArgs rng;
};

__device__ __forceinline__ float param(const void *p, int64_t i, int dtype, float none) {
    if (!p) return none;
    if (dtype == CT_F32) return ((const float *)p)[i];
    if (dtype == CT_F16) return __half2float(((const __half *)p)[i]);
    return __bfloat162float(((const __nv_bfloat16 *)p)[i]);
}

__device__ __forceinline__ void put_param(void *p, int64_t i, int dtype, float v) {
    if (dtype == CT_F32) ((float *)p)[i] = v;
    else if (dtype == CT_F16) ((__half *)p)[i] = __float2half_rn(v);
    else ((__nv_bfloat16 *)p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float sigmoid(float a) { return __fdividef(1.f, 1.f + __expf(-a)); }

template <int ACT>
__device__ __forceinline__ float act_value(float a) {
    if (ACT == CT_ACT_RELU) return a < 0.f ? 0.f : a;
    if (ACT == CT_ACT_SILU) return a * sigmoid(a);
    if (ACT == CT_ACT_GELU) return 0.5f * a * (1.f + erff(a * 0.70710678f));
    return a;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float a) {
    if (ACT == CT_ACT_RELU) return a > 0.f ? 1.f : 0.f;
    if (ACT == CT_ACT_SILU) {
        const float s = sigmoid(a);
        return s * (1.f + a * (1.f - s));
    }
    if (ACT == CT_ACT_GELU)
        return 0.5f * (1.f + erff(a * 0.70710678f)) + a * __expf(-0.5f * a * a) * 0.39894228f;
    return 1.f;
}

// One block's part of an image: a range of rows in one column tile.
struct Tile {
    int64_t n, part;       // image; chunk * ctiles + tile, the partials' index
    int64_t e0, e1, a0;    // the image's elements, and its start rounded down
    int head;
    int64_t r0, r1;        // rows
    int p0, p1;            // positions within a row
    int col;               // this thread's vector column
    int ty;
    bool on;

    __device__ __forceinline__ Tile(const GnGeom &g, int64_t item) {
        const int64_t per = (int64_t)g.chunks * g.ctiles;
        n = item / per;
        part = item - n * per;
        const int64_t chunk = part / g.ctiles;
        const int ct = (int)(part - chunk * g.ctiles);
        e0 = n * g.E;
        e1 = e0 + g.E;
        head = (int)(e0 & 7);
        a0 = e0 - head;
        r0 = chunk * g.rpc;
        r1 = r0 + g.rpc < g.rows ? r0 + g.rpc : g.rows;
        p0 = ct * g.bx * 8;
        p1 = p0 + g.bx * 8 < g.LV * 8 ? p0 + g.bx * 8 : g.LV * 8;
        const int tx = threadIdx.x % g.bx;
        ty = threadIdx.x / g.bx;
        col = ct * g.bx + tx;
        on = ty < g.by && col < g.LV;
    }
    __device__ __forceinline__ int channel0(const GnGeom &g) const {
        int c = (8 * col - head) % g.C;
        return c < 0 ? c + g.C : c;
    }
    __device__ __forceinline__ int64_t elem(const GnGeom &g, int64_t row) const {
        return a0 + 8 * (row * g.LV + col);
    }
    __device__ __forceinline__ uint32_t bits(int64_t e) const {   // which of e..e+7 are the image's
        if (e >= e0 && e + 8 <= e1) return 0xFFu;
        uint32_t m = 0;
        for (int k = 0; k < 8; ++k)
            if (e + k >= e0 && e + k < e1) m |= 1u << k;
        return m;
    }
};

__device__ __forceinline__ float group_sum(float v, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Merge (count, mean, M2) triples: `at(i, ...)` gives entry i of `n`; `lanes`
// threads share the work.  Mean first, then the distances from it.
template <typename F>
__device__ __forceinline__ void merge(int64_t n, int lane, int lanes, F at, float &cnt, float &mean, float &m2) {
    float sn = 0.f, sm = 0.f, c, m, q;
    for (int64_t i = lane; i < n; i += lanes) {
        at(i, c, m, q);
        if (c > 0.f) {
            sn += c;
            sm += c * m;
        }
    }
    sn = group_sum(sn, lanes);
    sm = group_sum(sm, lanes);
    cnt = sn;
    mean = sn > 0.f ? sm / sn : 0.f;
    float sq = 0.f;
    for (int64_t i = lane; i < n; i += lanes) {
        at(i, c, m, q);
        if (c > 0.f) {
            const float d = m - mean;
            sq += q + c * d * d;
        }
    }
    m2 = group_sum(sq, lanes);
}

// ---- forward ----------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(kThreads) gn_stats_kernel(const GnGeom g, const Params p) {
    __shared__ float sn[kThreads * 8], sm[kThreads * 8], sq[kThreads * 8];
    for (int64_t item = blockIdx.x; item < g.items; item += gridDim.x) {
        const Tile t(g, item);
        if (t.on) {
            float k0[8], s[8], ss[8], n[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) k0[k] = s[k] = ss[k] = n[k] = 0.f;
            for (int64_t r = t.r0 + t.ty; r < t.r1; r += g.by) {
                const int64_t e = t.elem(g, r);
                const uint32_t bits = t.bits(e);
                if (bits == 0) continue;
                float v[8];
                load8((const T *)p.x + e, bits, p.vec, v);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if ((bits >> k) & 1u) {
                        if (n[k] == 0.f) k0[k] = v[k];
                        const float d = v[k] - k0[k];
                        s[k] += d;
                        ss[k] += d * d;
                        n[k] += 1.f;
                    }
                }
            }
            const int at = (t.ty * g.bx + t.col) * 8 - t.p0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float inv = n[k] > 0.f ? 1.f / n[k] : 0.f;
                sn[at + k] = n[k];
                sm[at + k] = k0[k] + s[k] * inv;
                sq[at + k] = ss[k] - s[k] * s[k] * inv;
            }
        }
        __syncthreads();
        // groups: a power of two of lanes each
        int lanes = 1;
        while (lanes < 32 && lanes * 2 * g.G <= kThreads) lanes *= 2;
        const int per = kThreads / lanes, lane = threadIdx.x % lanes;
        const int width = g.bx * 8;
        for (int gb = 0; gb < g.G; gb += per) {
            const int gi = gb + threadIdx.x / lanes;
            const int each = g.Cg * g.wraps;
            float c, m, q;
            merge((int64_t)(gi < g.G ? each : 0) * g.by, lane, lanes,
                  [&](int64_t i, float &cn, float &mn, float &m2) {
                      const int y = (int)(i / each), j = (int)(i - (int64_t)y * each);
                      const int w = j / g.Cg, ch = gi * g.Cg + (j - w * g.Cg);
                      const int pos = (ch + t.head) % g.C + w * g.C;
                      cn = 0.f;
                      if (pos >= t.p0 && pos < t.p1) {
                          const int at = y * width + pos - t.p0;
                          cn = sn[at]; mn = sm[at]; m2 = sq[at];
                      }
                  }, c, m, q);
            if (gi < g.G && lane == 0) {
                float *out = p.part + ((t.n * g.chunks * g.ctiles + t.part) * g.G + gi) * 3;
                out[0] = c; out[1] = m; out[2] = q;
            }
        }
        __syncthreads();
    }
}

// One warp per (image, group): the partials' statistics joined.
__global__ void __launch_bounds__(kThreads) gn_finalize_kernel(const GnGeom g, const Params p) {
    const int64_t parts = (int64_t)g.chunks * g.ctiles, all = g.N * g.G;
    const int lane = threadIdx.x & 31;
    for (int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; w < all;
         w += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t n = w / g.G, gi = w - n * g.G;
        float c, m, q;
        merge(parts, lane, 32, [&](int64_t i, float &cn, float &mn, float &m2) {
            const float *in = p.part + ((n * parts + i) * g.G + gi) * 3;
            cn = in[0]; mn = in[1]; m2 = in[2];
        }, c, m, q);
        if (lane == 0) {
            const float var = q / fmaxf((float)((double)g.S * g.Cg), 1.f);
            p.mean[w] = m;
            p.rstd[w] = 1.f / sqrtf(var + p.eps);
        }
    }
}

template <typename T, int ACT, bool DROP>
__global__ void __launch_bounds__(kThreads) gn_apply_kernel(const GnGeom g, const Params p) {
    const Philox philox(p.rng);
    for (int64_t item = blockIdx.x; item < g.items; item += gridDim.x) {
        const Tile t(g, item);
        if (!t.on) continue;
        float mean[8], mul[8], add[8];
        int c = t.channel0(g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t at = t.n * g.G + c / g.Cg;
            mean[k] = p.mean[at];
            mul[k] = p.rstd[at] * param(p.weight, c, p.param_dtype, 1.f);
            add[k] = param(p.bias, c, p.param_dtype, 0.f);
            if (++c == g.C) c = 0;
        }
        for (int64_t r = t.r0 + t.ty; r < t.r1; r += g.by) {
            const int64_t e = t.elem(g, r);
            const uint32_t bits = t.bits(e);
            if (bits == 0) continue;
            float v[8];
            load8((const T *)p.x + e, bits, p.vec, v);
            uint32_t keep = 0xFFu;
            if (DROP) keep = keep_bits(philox((uint64_t)e >> 3), p.rng.threshold);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = act_value<ACT>((v[k] - mean[k]) * mul[k] + add[k]);
                if (DROP) v[k] = (keep >> k) & 1u ? v[k] * p.rng.scale : 0.f;
            }
            store8((T *)p.y + e, bits, p.vec, v);
        }
    }
}

// ---- backward ---------------------------------------------------------------

// A thread's eight channels: x - mean, its scale to a, and the shift.
struct Coef {
    float mean[8], mul[8], add[8];
    __device__ __forceinline__ void load(const GnGeom &g, const Params &p, const Tile &t) {
        int c = t.channel0(g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t at = t.n * g.G + c / g.Cg;
            mean[k] = p.mean[at];
            mul[k] = p.rstd[at] * param(p.weight, c, p.param_dtype, 1.f);
            add[k] = param(p.bias, c, p.param_dtype, 0.f);
            if (++c == g.C) c = 0;
        }
    }
};

// Per image, part and channel: sum da and sum da (x - mean).
template <typename T, int ACT, bool DROP>
__global__ void __launch_bounds__(kThreads) gn_back_sums_kernel(const GnGeom g, const Params p) {
    __shared__ float s0[kThreads * 8], s1[kThreads * 8];
    const Philox philox(p.rng);
    for (int64_t item = blockIdx.x; item < g.items; item += gridDim.x) {
        const Tile t(g, item);
        if (t.on) {
            Coef k8;
            k8.load(g, p, t);
            float u[8], w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = w[k] = 0.f;
            for (int64_t r = t.r0 + t.ty; r < t.r1; r += g.by) {
                const int64_t e = t.elem(g, r);
                const uint32_t bits = t.bits(e);
                if (bits == 0) continue;
                float v[8], d[8];
                load8((const T *)p.x + e, bits, p.vec, v);
                load8((const T *)p.dy + e, bits, p.vec, d);
                uint32_t keep = bits;
                if (DROP) keep &= keep_bits(philox((uint64_t)e >> 3), p.rng.threshold);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float xc = v[k] - k8.mean[k];
                    const float da = (keep >> k) & 1u
                        ? (DROP ? d[k] * p.rng.scale : d[k]) * act_slope<ACT>(xc * k8.mul[k] + k8.add[k]) : 0.f;
                    u[k] += da;
                    // a dropped element adds nothing, whatever x holds there
                    w[k] += (keep >> k) & 1u ? da * xc : 0.f;
                }
            }
            const int at = (t.ty * g.bx + t.col) * 8 - t.p0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s0[at + k] = u[k];
                s1[at + k] = w[k];
            }
        }
        __syncthreads();
        const int width = g.bx * 8;
        for (int c = threadIdx.x; c < g.C; c += kThreads) {
            float u = 0.f, w = 0.f;
            for (int j = 0; j < g.wraps; ++j) {
                const int pos = (c + t.head) % g.C + j * g.C;
                if (pos < t.p0 || pos >= t.p1) continue;
                for (int y = 0; y < g.by; ++y) {
                    u += s0[y * width + pos - t.p0];
                    w += s1[y * width + pos - t.p0];
                }
            }
            float *out = p.part + ((t.n * g.chunks * g.ctiles + t.part) * g.C + c) * 2;
            out[0] = u;
            out[1] = w;
        }
        __syncthreads();
    }
}

// One block per (image, group): the channels' sums joined over the parts
// (kept for dw and db) and the group's two means.
__global__ void __launch_bounds__(kThreads) gn_back_finalize_kernel(const GnGeom g, const Params p) {
    __shared__ float r0[kThreads / 32], r1[kThreads / 32];
    const int64_t parts = (int64_t)g.chunks * g.ctiles, all = g.N * g.G;
    for (int64_t item = blockIdx.x; item < all; item += gridDim.x) {
        const int64_t n = item / g.G;
        const int gi = (int)(item - n * g.G);
        const float rstd = p.rstd[item];
        float m0 = 0.f, m1 = 0.f;
        for (int j = threadIdx.x; j < g.Cg; j += kThreads) {
            const int c = gi * g.Cg + j;
            float u = 0.f, w = 0.f;
            for (int64_t i = 0; i < parts; ++i) {
                const float *in = p.part + ((n * parts + i) * g.C + c) * 2;
                u += in[0];
                w += in[1];
            }
            w *= rstd;
            p.sums[(n * g.C + c) * 2] = u;
            p.sums[(n * g.C + c) * 2 + 1] = w;
            const float wt = param(p.weight, c, p.param_dtype, 1.f);
            m0 += wt * u;
            m1 += wt * w;
        }
        m0 = group_sum(m0, 32);
        m1 = group_sum(m1, 32);
        if ((threadIdx.x & 31) == 0) {
            r0[threadIdx.x / 32] = m0;
            r1[threadIdx.x / 32] = m1;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            m0 = m1 = 0.f;
            for (int i = 0; i < kThreads / 32; ++i) {
                m0 += r0[i];
                m1 += r1[i];
            }
            const float inv = 1.f / fmaxf((float)((double)g.S * g.Cg), 1.f);
            p.coef[item * 2] = m0 * inv;
            p.coef[item * 2 + 1] = m1 * inv;
        }
        __syncthreads();
    }
}

// One warp per channel: dw and db, the images' sums joined.
__global__ void __launch_bounds__(kThreads) gn_back_params_kernel(const GnGeom g, const Params p) {
    const int lane = threadIdx.x & 31;
    for (int64_t c = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; c < g.C;
         c += (int64_t)gridDim.x * (kThreads / 32)) {
        float u = 0.f, w = 0.f;
        for (int64_t n = lane; n < g.N; n += 32) {
            u += p.sums[(n * g.C + c) * 2];
            w += p.sums[(n * g.C + c) * 2 + 1];
        }
        u = group_sum(u, 32);
        w = group_sum(w, 32);
        if (lane == 0) {
            if (p.dbias) put_param(p.dbias, c, p.param_dtype, u);
            if (p.dweight) put_param(p.dweight, c, p.param_dtype, w);
        }
    }
}

template <typename T, int ACT, bool DROP>
__global__ void __launch_bounds__(kThreads) gn_back_apply_kernel(const GnGeom g, const Params p) {
    const Philox philox(p.rng);
    for (int64_t item = blockIdx.x; item < g.items; item += gridDim.x) {
        const Tile t(g, item);
        if (!t.on) continue;
        Coef k8;
        k8.load(g, p, t);
        float m0[8], m1[8];   // rstd * mean(dh), rstd^2 * mean(dh h)
        int c = t.channel0(g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t at = t.n * g.G + c / g.Cg;
            const float rstd = p.rstd[at];
            m0[k] = rstd * p.coef[2 * at];
            m1[k] = rstd * rstd * p.coef[2 * at + 1];
            if (++c == g.C) c = 0;
        }
        for (int64_t r = t.r0 + t.ty; r < t.r1; r += g.by) {
            const int64_t e = t.elem(g, r);
            const uint32_t bits = t.bits(e);
            if (bits == 0) continue;
            float v[8], d[8];
            load8((const T *)p.x + e, bits, p.vec, v);
            load8((const T *)p.dy + e, bits, p.vec, d);
            uint32_t keep = 0xFFu;
            if (DROP) keep = keep_bits(philox((uint64_t)e >> 3), p.rng.threshold);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float xc = v[k] - k8.mean[k];
                const float da = (keep >> k) & 1u
                    ? (DROP ? d[k] * p.rng.scale : d[k]) * act_slope<ACT>(xc * k8.mul[k] + k8.add[k]) : 0.f;
                v[k] = da * k8.mul[k] - m0[k] - xc * m1[k];
            }
            store8((T *)p.dx + e, bits, p.vec, v);
        }
    }
}

// ---- host -------------------------------------------------------------------

constexpr int64_t kGridCap = 148 * 64;

int grid_for(int64_t n) { return (int)(n < 1 ? 1 : n < kGridCap ? n : kGridCap); }

template <int V>
struct Int {
    static constexpr int value = V;
};

template <typename F>
void by_act(int act, bool drop, F f) {
    if (drop) {
        if (act == CT_ACT_RELU) f(Int<CT_ACT_RELU>(), Int<1>());
        else if (act == CT_ACT_SILU) f(Int<CT_ACT_SILU>(), Int<1>());
        else if (act == CT_ACT_GELU) f(Int<CT_ACT_GELU>(), Int<1>());
        else f(Int<CT_ACT_IDENTITY>(), Int<1>());
    } else {
        if (act == CT_ACT_RELU) f(Int<CT_ACT_RELU>(), Int<0>());
        else if (act == CT_ACT_SILU) f(Int<CT_ACT_SILU>(), Int<0>());
        else if (act == CT_ACT_GELU) f(Int<CT_ACT_GELU>(), Int<0>());
        else f(Int<CT_ACT_IDENTITY>(), Int<0>());
    }
}

Params params_of(const GnArgs &a) {
    Params p = {};
    p.x = a.x; p.dy = a.dy; p.weight = a.weight; p.bias = a.bias;
    p.y = a.y; p.dx = a.dx; p.dweight = a.dweight; p.dbias = a.dbias;
    p.mean = a.mean; p.rstd = a.rstd;
    p.eps = a.eps;
    p.param_dtype = a.param_dtype;
    p.rng = a.rng;
    p.vec = (((uintptr_t)a.x | (uintptr_t)a.dy | (uintptr_t)a.y | (uintptr_t)a.dx) & 15) == 0;
    return p;
}

template <typename T>
ct_status forward_t(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    Params p = params_of(a);
    p.part = a.ws;
    const int grid = grid_for(g.items);
    gn_stats_kernel<T><<<grid, kThreads, 0, st>>>(g, p);
    gn_finalize_kernel<<<grid_for(ceil_div(g.N * g.G, kThreads / 32)), kThreads, 0, st>>>(g, p);
    by_act(a.act, a.drop, [&](auto act, auto drop) {
        gn_apply_kernel<T, decltype(act)::value, decltype(drop)::value != 0><<<grid, kThreads, 0, st>>>(g, p);
    });
    return launch_status();
}

template <typename T>
ct_status backward_t(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    Params p = params_of(a);
    p.part = a.ws;
    p.sums = p.part + g.items * g.C * 2;
    p.coef = p.sums + g.N * g.C * 2;
    const int grid = grid_for(g.items);
    by_act(a.act, a.drop, [&](auto act, auto drop) {
        gn_back_sums_kernel<T, decltype(act)::value, decltype(drop)::value != 0><<<grid, kThreads, 0, st>>>(g, p);
    });
    gn_back_finalize_kernel<<<grid_for(g.N * g.G), kThreads, 0, st>>>(g, p);
    if (a.dweight || a.dbias)
        gn_back_params_kernel<<<grid_for(ceil_div(g.C, kThreads / 32)), kThreads, 0, st>>>(g, p);
    if (a.dx)
        by_act(a.act, a.drop, [&](auto act, auto drop) {
            gn_back_apply_kernel<T, decltype(act)::value, decltype(drop)::value != 0><<<grid, kThreads, 0, st>>>(g, p);
        });
    return launch_status();
}

}  // namespace

GnGeom gn_geom(int64_t N, int64_t S, int64_t C, int64_t G) {
    GnGeom g = {};
    g.N = N; g.S = S; g.E = S * C;
    g.C = (int32_t)C; g.G = (int32_t)G; g.Cg = (int32_t)(C / G);
    int64_t d = C % 8 == 0 ? 8 : C % 4 == 0 ? 4 : C % 2 == 0 ? 2 : 1;
    g.wraps = (int32_t)(8 / d);
    g.LV = (int32_t)(C / d);
    // the head of an image whose elements do not start at a multiple of eight
    // can take one more row
    const int64_t head = g.E % 8 == 0 || N <= 1 ? 0 : 7;
    g.rows = ceil_div(head + g.E, (int64_t)g.LV * 8);
    g.ctiles = (int32_t)ceil_div(g.LV, kThreads);
    g.bx = (int32_t)ceil_div(g.LV, g.ctiles);
    int64_t by = kThreads / g.bx;
    if (by > g.rows) by = g.rows < 1 ? 1 : g.rows;
    g.by = (int32_t)by;
    // about four blocks per SM, each with eight rows or more per thread
    const int64_t tiles = N * g.ctiles < 1 ? 1 : N * g.ctiles;
    int64_t chunks = ceil_div(148 * 4, tiles);
    const int64_t most = ceil_div(g.rows, (int64_t)g.by * 8);
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    g.rpc = ceil_div(g.rows < 1 ? 1 : g.rows, chunks);
    g.chunks = (int32_t)ceil_div(g.rows < 1 ? 1 : g.rows, g.rpc);
    g.items = N * g.chunks * g.ctiles;
    return g;
}

size_t gn_forward_ws(const GnGeom &g) {
    return (size_t)(g.items * g.G * 3) * sizeof(float) + (size_t)(2 * g.N * g.G) * sizeof(float);
}

size_t gn_backward_ws(const GnGeom &g) {
    return (size_t)(g.items * g.C * 2 + g.N * g.C * 2 + g.N * g.G * 2) * sizeof(float);
}

ct_status gn_forward(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    GnArgs b = a;
    // statistics that the caller does not want live behind the partials
    float *own = a.ws + g.items * g.G * 3;
    if (!b.mean) b.mean = own;
    if (!b.rstd) b.rstd = own + g.N * g.G;
    if (a.dtype == CT_F32) return forward_t<float>(g, b, st);
    if (a.dtype == CT_F16) return forward_t<__half>(g, b, st);
    return forward_t<__nv_bfloat16>(g, b, st);
}

ct_status gn_backward(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    if (a.dtype == CT_F32) return backward_t<float>(g, a, st);
    if (a.dtype == CT_F16) return backward_t<__half>(g, a, st);
    return backward_t<__nv_bfloat16>(g, a, st);
}

}  // namespace ct
