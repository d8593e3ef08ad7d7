// Rotary positions of several axes: pair (a, b) of a head at pixel s becomes
//
//     (a cos t - b sin t, a sin t + b cos t),   t = position of s on the pair's axis * the pair's frequency.
//
// Bound: HBM, x in and y out.  A thread has the pairs of one vector (or of two,
// one in each half of the head) of one pixel, makes their sines and cosines
// once and walks the heads with them in registers.  The angle is formed in
// turns in 64 bits, where a position of 2^31 still keeps its fraction of a
// turn to 2^-22, reduced to half a turn and rounded; sincospi takes it from
// there.  That is some 40 operations a pair, for all heads together.
#include <type_traits>

#include "ct_cuda_util.h"
#include "rotary.h"
#include "vec16.cuh"

namespace ct {

namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 4;        // of a thread, in flight

// E elements as they are loaded: a 16-byte vector, or one element.
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

// The position of pixel s of image n on each axis.
__device__ __forceinline__ void positions_of(const RotaryParams &p, int64_t n, int64_t s, double (&at)[3]) {
    at[0] = at[1] = at[2] = 0.0;
    if (p.pos_type == CT_POSITION_GRID) {
        if (p.S <= 0xFFFFFFFFll) {
            uint32_t r = (uint32_t)s;
#pragma unroll
            for (int a = 2; a > 0; --a)
                if (a < p.axes) {
                    const uint32_t q = r / (uint32_t)p.grid[a];
                    at[a] = (double)(r - q * (uint32_t)p.grid[a]);
                    r = q;
                }
            at[0] = (double)r;
        } else {
#pragma unroll
            for (int a = 2; a > 0; --a)
                if (a < p.axes) {
                    at[a] = (double)(s % p.grid[a]);
                    s /= p.grid[a];
                }
            at[0] = (double)s;
        }
        return;
    }
    const int64_t i = n * p.pos_image + s * p.axes;
#pragma unroll
    for (int a = 0; a < 3; ++a)
        if (a < p.axes) {
            if (p.pos_type == CT_POSITION_I32) at[a] = (double)((const int32_t *)p.positions)[i + a];
            else if (p.pos_type == CT_POSITION_I64) at[a] = (double)((const int64_t *)p.positions)[i + a];
            else at[a] = (double)((const float *)p.positions)[i + a];
        }
}

// E: elements of a vector (1: none).  An item of a head is
//   HALVES: E pairs, whose two sides lie rot / 2 apart; behind them E elements
//           that stay as they are;
//   else:   a vector of E / 2 pairs, some of which may stay (E = 1: one pair,
//           behind them one element that stays).
template <typename T, int E, bool HALVES>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    constexpr int P = HALVES || E == 1 ? E : E / 2;     // pairs of an item
    constexpr bool kTwo = HALVES || E == 1;             // two loads
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= p.threads) return;
    int64_t row;
    int item, group;
    if (p.threads <= 0xFFFFFFFFll) {
        const uint32_t r = (uint32_t)id / (uint32_t)p.items;
        item = (int)((uint32_t)id - r * (uint32_t)p.items);
        row = r / (uint32_t)p.groups;
        group = (int)(r - (uint32_t)row * (uint32_t)p.groups);
    } else {
        const int64_t r = id / p.items;
        item = (int)(id - r * p.items);
        row = r / p.groups;
        group = (int)(r - row * p.groups);
    }
    const int64_t n = row / p.S, s = row - n * p.S;
    const int half = p.rot / 2, turned = kTwo ? half / E : (p.rot + E - 1) / E;    // items with a pair that turns
    const int first = item * P;                       // pair
    const bool turns = item < turned;
    float c[P], d[P];
    double where[3];
    positions_of(p, n, s, where);
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int q = first + j;
        if (turns && q < half) {
            double t = where[0];
            if (p.axes > 1 && q >= p.first[1]) t = where[1];
            if (p.axes > 2 && q >= p.first[2]) t = where[2];
            t *= p.turns[q];
            sincospif(2.f * (float)(t - rint(t)), &d[j], &c[j]);
            d[j] *= p.sign;
        }
    }
    // where the item's elements are in a head
    const int64_t at = turns ? (HALVES ? (int64_t)first : E == 1 ? 2 * (int64_t)first : (int64_t)item * E)
                             : kTwo ? p.rot + (int64_t)(item - turned) * E : (int64_t)item * E;
    const int64_t over = HALVES ? half : 1;
    const T *x = (const T *)p.x + n * p.xs[0] + s * p.xs[1] + at;
    T *y = (T *)p.y + n * p.ys[0] + s * p.ys[1] + at;
    const int64_t h0 = (int64_t)group * p.per, h1 = h0 + p.per < p.H ? h0 + p.per : p.H;
    for (int64_t h = h0; h < h1; h += kHeads) {
        Raw<T, E> ra[kHeads], rb[kTwo ? kHeads : 1];
#pragma unroll
        for (int u = 0; u < kHeads; ++u)
            if (h + u < h1) {
                ra[u] = load_raw<T, E>(x + (h + u) * p.xs[2]);
                if constexpr (kTwo)
                    if (turns) rb[u] = load_raw<T, E>(x + (h + u) * p.xs[2] + over);
            }
#pragma unroll
        for (int u = 0; u < kHeads; ++u)
            if (h + u < h1) {
                T *out = y + (h + u) * p.ys[2];
                float a[E], b[E];
                of_raw<T, E>(ra[u], a);
                if constexpr (kTwo) {
                    if (turns) {
                        of_raw<T, E>(rb[u], b);
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const float v = a[j], w = b[j];
                            a[j] = fmaf(v, c[j], -(w * d[j]));
                            b[j] = fmaf(v, d[j], w * c[j]);
                        }
                        store_e<T, E>(out + over, b);
                    }
                } else if (turns) {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        if (first + j < half) {
                            const float v = a[2 * j], w = a[2 * j + 1];
                            a[2 * j] = fmaf(v, c[j], -(w * d[j]));
                            a[2 * j + 1] = fmaf(v, d[j], w * c[j]);
                        }
                }
                store_e<T, E>(out, a);
            }
    }
}

template <typename T, int E, bool HALVES>
ct_status launch(RotaryParams &p, cudaStream_t st) {
    const int64_t half = p.rot / 2;
    p.items = (int32_t)(HALVES || E == 1 ? half / E + (p.D - p.rot) / E : p.D / E);
    // as many heads a thread as leave 2048 threads an SM
    const int64_t threads = p.N * p.S * p.items, enough = 148 * 2048;
    int64_t groups = ceil_div(enough, threads);
    if (groups > p.H) groups = p.H;
    p.per = (int32_t)ceil_div(p.H, groups);
    p.groups = (int32_t)ceil_div(p.H, (int64_t)p.per);
    p.threads = threads * p.groups;
    const int64_t blocks = ceil_div(p.threads, (int64_t)kThreads);
    if (blocks > 0x7FFFFFFF) return CT_ERR_ATTR;
    rotary_kernel<T, E, HALVES><<<(unsigned)blocks, kThreads, 0, st>>>(p);
    return launch_status();
}

template <typename T>
ct_status run(int pairs, RotaryParams &p, cudaStream_t st) {
    constexpr int V = kVec<T>;
    bool vec = (((uintptr_t)p.x | (uintptr_t)p.y) & 15) == 0 && p.D % V == 0;
    const int64_t sizes[3] = {p.N, p.S, p.H};
    for (int a = 0; a < 3; ++a) vec = vec && (sizes[a] == 1 || (p.xs[a] % V == 0 && p.ys[a] % V == 0));
    if (pairs == CT_PAIRS_HALVES) {
        if (vec && p.rot / 2 % V == 0) return launch<T, V, true>(p, st);
        return launch<T, 1, true>(p, st);
    }
    return vec ? launch<T, V, false>(p, st) : launch<T, 1, false>(p, st);
}

}  // namespace

ct_status rotary_run(int dtype, int pairs, RotaryParams &p, cudaStream_t st) {
    if (dtype == CT_F32) return run<float>(pairs, p, st);
    if (dtype == CT_F16) return run<__half>(pairs, p, st);
    return run<__nv_bfloat16>(pairs, p, st);
}

}  // namespace ct
