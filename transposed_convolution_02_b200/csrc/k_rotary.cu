// Rotary positions of several axes: pair (a, b) of a head at pixel s becomes
//
//     (a cos t - b sin t, a sin t + b cos t),   t = position of s on the pair's axis * the pair's frequency.
//
// Bound: HBM, x in and y out.  A thread has the pairs of one vector (or of two,
// one in each half of the head) of one pixel, makes their sines and cosines
// once and walks the heads (or images) with them in registers.  The angle is formed in
// turns.  A position of up to 24 bits times a frequency of two floats (48 bits)
// is formed in fp32: the product's rounding is known exactly (fused
// multiply-add), and so is what whole and quarter turns leave of it; the rounding
// joins that remainder, an eighth of a turn at most, once it is an angle.  Sines
// and cosines come out to 1.5 * 2^-24 for positions below 2^17 (2^-45 of the
// angle is lost beside that, at most).  Larger positions, and frequencies above a
// turn a position, are multiplied in 64 bits and reduced alike.
// Measured (GPU time; against the measured copy rate): [2,16x32x32,24,128] bf16
// 65 us (0.95; 185 with angles in 64 bits and divisions for every pair),
// [3,57x91,5,72] fp32 10.5 (0.65: two rounds of blocks), one head of 64 at
// [16,64x64x16] bf16 44 (0.93: the images share the angles), heads of 72 with
// sides 35 apart 60 (0.57: single elements).
#include <type_traits>
#include <utility>

#include "ct_cuda_util.h"
#include "rotary.h"
#include "vec16.cuh"

namespace ct {

namespace {

constexpr int kThreads = 128;

// Heads of a thread in flight: short vectors need more of them for the same bytes.
template <int E>
constexpr int kHeads = E <= 2 ? 8 : 4;

// E elements as they are loaded: one word of 2 to 16 bytes.
template <int BYTES>
struct Word;
template <>
struct Word<2> { using type = uint16_t; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };
template <typename T, int E>
using Raw = typename Word<E * sizeof(T)>::type;

template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_raw(const T *p) {
    return *reinterpret_cast<const Raw<T, E> *>(p);
}

template <typename T, int E>
__device__ __forceinline__ void of_raw(const Raw<T, E> &r, float (&f)[E]) {
    if constexpr (E == 1) {
        f[0] = to_f<T>(*reinterpret_cast<const T *>(&r));
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < E; ++j) f[j] = __uint_as_float(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float2 v = unpack1(w[j], T());
                f[2 * j] = v.x, f[2 * j + 1] = v.y;
            }
        }
    }
}

template <typename T, int E>
__device__ __forceinline__ void store_e(T *p, const float (&f)[E]) {
    if constexpr (E == 1) {
        *p = from_f<T>(f[0]);
    } else {
        Raw<T, E> r;
        uint32_t *w = reinterpret_cast<uint32_t *>(&r);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < E; ++j) w[j] = __float_as_uint(f[j]);
        } else {
#pragma unroll
            for (int j = 0; j < E / 2; ++j) w[j] = pack1(make_float2(f[2 * j], f[2 * j + 1]), T());
        }
        *reinterpret_cast<Raw<T, E> *>(p) = r;
    }
}

// The position of pixel s of image n on each axis, as a float and, where that
// does not hold it, in 64 bits.
struct Positions {
    float near[3];
    double far[3];
    bool is_far;
};

__device__ __forceinline__ void positions_of(const RotaryParams &p, int64_t n, int64_t s, Positions &at) {
    at.is_far = false;
    at.near[0] = at.near[1] = at.near[2] = 0.f;
    if (p.pos_type == CT_POSITION_GRID && p.small && p.small_grid) {
        int rest = (int)s;
#pragma unroll
        for (int a = 2; a > 0; --a)
            if (a < p.axes) {
                const int q = divq(rest, p.by_grid[a]);
                at.near[a] = (float)(rest - q * (int)p.grid[a]);
                rest = q;
            }
        at.near[0] = (float)rest;
        return;
    }
    if (p.pos_type == CT_POSITION_F32) {
        const float *from = (const float *)p.positions + n * p.pos_image + s * p.axes;
#pragma unroll
        for (int a = 0; a < 3; ++a) {
            if (a < p.axes) at.near[a] = from[a];
            if (fabsf(at.near[a]) > p.near) at.is_far = true;
            at.far[a] = (double)at.near[a];
        }
        return;
    }
    int64_t whole[3] = {0, 0, 0};
    if (p.pos_type == CT_POSITION_GRID) {
#pragma unroll
        for (int a = 2; a > 0; --a)
            if (a < p.axes) {
                const int64_t q = s / p.grid[a];
                whole[a] = s - q * p.grid[a];
                s = q;
            }
        whole[0] = s;
    } else {
        const int64_t i = n * p.pos_image + s * p.axes;
#pragma unroll
        for (int a = 0; a < 3; ++a)
            if (a < p.axes)
                whole[a] = p.pos_type == CT_POSITION_I32 ? ((const int32_t *)p.positions)[i + a]
                                                         : ((const int64_t *)p.positions)[i + a];
    }
#pragma unroll
    for (int a = 0; a < 3; ++a) {
        at.near[a] = (float)whole[a];
        if (fabsf(at.near[a]) > p.near || whole[a] > 16777216 || whole[a] < -16777216) at.is_far = true;
    }
    if (at.is_far)
        for (int a = 0; a < 3; ++a) at.far[a] = (double)whole[a];
}

__device__ __forceinline__ float2 twice(float f) { return make_float2(f, f); }

// Two angles in turns, without whole ones: `high`, at most half a turn, which
// holds all its bits, and what it lacks.
struct Turns {
    float2 high, low;
};

// Their cosines and sines: the nearest quarter turn is taken off, and Taylor's
// polynomials serve what is left, an eighth of a turn at most (the first terms
// left out are below 2^-29).  Adding 3 * 2^22 rounds to a whole number of
// quarters, which then are the sum's last bits.
__device__ __forceinline__ void turn(const Turns &t, float2 &c, float2 &s) {
    const float2 z = __ffma2_rn(__fadd2_rn(t.high, t.low), twice(4.f), twice(12582912.f));
    const float2 g = __ffma2_rn(__fadd2_rn(z, twice(-12582912.f)), twice(-0.25f), t.high);      // exact; beside a border to 2^-28
    // 2 pi in two floats
    const float2 rest = __ffma2_rn(g, twice(-1.7484556e-7f), __fmul2_rn(t.low, twice(6.2831855f)));
    const float2 x = __ffma2_rn(g, twice(6.2831855f), rest), q = __fmul2_rn(x, x);
    float2 a = __ffma2_rn(q, twice(1.f / 362880), twice(-1.f / 5040));
    a = __ffma2_rn(a, q, twice(1.f / 120));
    a = __ffma2_rn(a, q, twice(-1.f / 6));
    a = __ffma2_rn(__fmul2_rn(a, q), x, x);
    float2 b = __ffma2_rn(q, twice(-1.f / 3628800), twice(1.f / 40320));
    b = __ffma2_rn(b, q, twice(-1.f / 720));
    b = __ffma2_rn(b, q, twice(1.f / 24));
    b = __ffma2_rn(b, q, twice(-0.5f));
    b = __ffma2_rn(b, q, twice(1.f));
    auto place = [](uint32_t n, float sine, float cosine, float &to_c, float &to_s) {
        const bool odd = n & 1;
        const uint32_t high = n << 30, both = high ^ n << 31;      // bit 1 of n, and of n + 1, on top
        to_s = __uint_as_float((high & 0x80000000u) ^ __float_as_uint(odd ? cosine : sine));
        to_c = __uint_as_float((both & 0x80000000u) ^ __float_as_uint(odd ? sine : cosine));
    };
    place(__float_as_uint(z.x), a.x, b.x, c.x, s.x);
    place(__float_as_uint(z.y), a.y, b.y, c.y, s.y);
}

// Positions times frequencies (as high and low parts).
__device__ __forceinline__ Turns turns_of(float2 pos, float2 hi, float2 lo) {
    const float2 t = __fmul2_rn(pos, hi), minus = make_float2(-t.x, -t.y);
    const float2 rest = __ffma2_rn(pos, lo, __ffma2_rn(pos, hi, minus));
    const float2 whole = __fadd2_rn(__fadd2_rn(t, twice(12582912.f)), twice(-12582912.f));
    return {__fadd2_rn(t, make_float2(-whole.x, -whole.y)), rest};
}

// A product in 64 bits.
__device__ __forceinline__ void turns_of(double t, float &high, float &low) {
    t -= rint(t);
    high = (float)t;
    low = (float)(t - (double)high);
}

// E: elements of a vector.  An item of a head is
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
    int64_t row, n, s;
    int item, group;
    if (p.small) {
        const int r = divq((int)id, p.by_items), w = divq(r, p.by_groups), im = divq(w, p.by_s);
        item = (int)id - r * p.items;
        group = r - w * p.groups;
        row = w;
        n = im;
        s = w - im * (int)p.S;
    } else {
        const int64_t r = id / p.items;
        item = (int)(id - r * p.items);
        row = r / p.groups;
        group = (int)(r - row * p.groups);
        n = row / p.S;
        s = row - n * p.S;
    }
    const int half = p.rot / 2, turned = kTwo ? half / E : (p.rot + E - 1) / E;    // items with a pair that turns
    const int first = item * P;                       // pair
    const bool turns = item < turned;
    constexpr int Q = (P + 1) / 2;
    float2 cs[Q], sn[Q];                              // two pairs together
    if (turns) {
        Positions where;
        positions_of(p, n, s, where);
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            const int q = first + 2 * j;
            // P is even, but for single elements, whose second pair is no one's
            const float4 f = P > 1 ? *reinterpret_cast<const float4 *>(p.parts[q])
                                   : make_float4(p.parts[q][0], p.parts[q][1], 0.f, 0.f);
            auto axis = [&](int i) { return p.axes > 1 && i >= p.first[1] ? p.axes > 2 && i >= p.first[2] ? 2 : 1 : 0; };
            const int a0 = axis(q), a1 = axis(q + 1);
            Turns r;
            if (!where.is_far) {
                const float2 pos = make_float2(a0 == 2 ? where.near[2] : a0 == 1 ? where.near[1] : where.near[0],
                                               a1 == 2 ? where.near[2] : a1 == 1 ? where.near[1] : where.near[0]);
                r = turns_of(pos, make_float2(f.x, f.z), make_float2(f.y, f.w));
            } else {
                turns_of((a0 == 2 ? where.far[2] : a0 == 1 ? where.far[1] : where.far[0]) * p.turns[q], r.high.x, r.low.x);
                turns_of(P == 1 ? 0.0 : (a1 == 2 ? where.far[2] : a1 == 1 ? where.far[1] : where.far[0]) * p.turns[q + 1],
                         r.high.y, r.low.y);
            }
            turn(r, cs[j], sn[j]);
            sn[j] = __fmul2_rn(sn[j], twice(p.sign));
        }
    }
    auto c = [&](int j) { return j & 1 ? cs[j / 2].y : cs[j / 2].x; };
    auto d = [&](int j) { return j & 1 ? sn[j / 2].y : sn[j / 2].x; };
    // where the item's elements are in a head
    const int64_t at = turns ? (HALVES ? (int64_t)first : E == 1 ? 2 * (int64_t)first : (int64_t)item * E)
                             : kTwo ? p.rot + (int64_t)(item - turned) * E : (int64_t)item * E;
    const int64_t over = HALVES ? half : 1;
    const T *x = (const T *)p.x + n * p.xs[0] + s * p.xs[1] + at;
    T *y = (T *)p.y + n * p.ys[0] + s * p.ys[1] + at;
    const int64_t h0 = (int64_t)group * p.per;
    int left = p.H - h0 < p.per ? (int)(p.H - h0) : p.per;
    x += h0 * p.xs[2];
    y += h0 * p.ys[2];
    const int64_t xh = p.xs[2], yh = p.ys[2];
    // the next heads: all U of them there, or the `left` last ones
    auto heads = [&](auto all) {
        constexpr bool ALL = decltype(all)::value;
        constexpr int U = kHeads<E>;
        Raw<T, E> ra[U], rb[kTwo ? U : 1];
        const T *from = x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!ALL && u >= left) break;
            ra[u] = load_raw<T, E>(from);
            if constexpr (kTwo)
                if (turns) rb[u] = load_raw<T, E>(from + over);
            from += xh;
        }
        x = from;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!ALL && u >= left) break;
            float a[E], b[E];
            of_raw<T, E>(ra[u], a);
            if constexpr (kTwo) {
                if (turns) {
                    of_raw<T, E>(rb[u], b);
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        const float v = a[j], w = b[j];
                        a[j] = fmaf(v, c(j), -(w * d(j)));
                        b[j] = fmaf(v, d(j), w * c(j));
                    }
                    store_e<T, E>(y + over, b);
                }
            } else if (turns) {
#pragma unroll
                for (int j = 0; j < P; ++j)
                    if (first + j < half) {
                        const float v = a[2 * j], w = a[2 * j + 1];
                        a[2 * j] = fmaf(v, c(j), -(w * d(j)));
                        a[2 * j + 1] = fmaf(v, d(j), w * c(j));
                    }
            }
            store_e<T, E>(y, a);
            y += yh;
        }
    };
    for (; left >= kHeads<E>; left -= kHeads<E>) heads(std::true_type());
    if (left > 0) heads(std::false_type());
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
    p.small = p.threads < 0x7FFFFFFF;
    if (p.small) {
        p.by_items = make_magic((uint32_t)p.items);
        p.by_groups = make_magic((uint32_t)p.groups);
        p.by_s = make_magic((uint32_t)p.S);
        for (int a = 0; a < p.axes; ++a) p.by_grid[a] = make_magic((uint32_t)p.grid[a]);
    }
    const int64_t blocks = ceil_div(p.threads, (int64_t)kThreads);
    if (blocks > 0x7FFFFFFF) return CT_ERR_ATTR;
    rotary_kernel<T, E, HALVES><<<(unsigned)blocks, kThreads, 0, st>>>(p);
    return launch_status();
}

// The longest vectors that every head, and every side of its pairs, can be cut
// into.
template <typename T, int E>
ct_status run(int pairs, RotaryParams &p, cudaStream_t st) {
    bool fits = (((uintptr_t)p.x | (uintptr_t)p.y) & (E * sizeof(T) - 1)) == 0 && p.D % E == 0;
    const int64_t sizes[3] = {p.N, p.S, p.H};
    for (int a = 0; a < 3; ++a) fits = fits && (sizes[a] == 1 || (p.xs[a] % E == 0 && p.ys[a] % E == 0));
    if (pairs == CT_PAIRS_HALVES) fits = fits && p.rot / 2 % E == 0;
    if constexpr (E > 1)
        if (!fits) return run<T, E / 2>(pairs, p, st);
    return pairs == CT_PAIRS_HALVES ? launch<T, E, true>(p, st) : launch<T, E, false>(p, st);
}

}  // namespace

ct_status rotary_run(int dtype, int pairs, RotaryParams &p, cudaStream_t st) {
    // Images whose positions are the same share angles as heads do: where heads
    // are few, a thread walks the images ([16,64x64x16,1,64] bf16 44 us, 97 with
    // each image's angles made again).
    if (p.H < kHeads<8> && p.N > p.H && p.N < 1 << 24 && (p.pos_type == CT_POSITION_GRID || p.pos_image == 0)) {
        std::swap(p.N, p.H);
        std::swap(p.xs[0], p.xs[2]);
        std::swap(p.ys[0], p.ys[2]);
    }
    if (dtype == CT_F32) return run<float, 4>(pairs, p, st);
    if (dtype == CT_F16) return run<__half, 8>(pairs, p, st);
    return run<__nv_bfloat16, 8>(pairs, p, st);
}

}  // namespace ct
