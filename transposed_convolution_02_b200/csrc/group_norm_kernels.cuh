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
// Bound: HBM, at x and y once forward, x, dy and dx once backward.  All of a
// group's values are needed before its first output, so there are two passes over
// the inputs, of which the second finds them in L2 or reads HBM again.
//   One launch: a cluster of blocks works on an image (a strip), joins its
// blocks' sums through distributed shared memory and goes on to the second
// pass.  For small tensors, where a launch counts, and where such clusters fill
// the GPU.
//   Two launches else: sums, with a part of them from every block in the
// workspace, and apply, each block joining the parts of its groups.  The
// second starts while the first one ends (programmatic dependent launch).
// Inputs of up to about 90 MB are then found in L2.
// Measured, [8, 128x128, 128] fp16 with SiLU, 33.5 MB in and out: 25.4 us,
// where reading x alone takes 6.9 and copying it 12.3.  [16, 16384, 256] fp32,
// 268 MB in and out: 148 us, where x is read twice from HBM; one read and one
// write of it would take 82 at the measured copy rate (a copy takes 87).
// Tried and slower: images taken in waves that fit L2 (every wave paid the 10
// us that do not stream; vocoder size 176 to 230 us), a ring of bulk copies
// with a copying warp (its hand-overs cost more than the registers it saved),
// clusters of 8 whole-SM blocks or of 16 (placed slowly), a second pass with
// rows handed out by a counter (a barrier for each piece; 27.1 us) or in
// reverse (no change), streaming stores (no change).
//
// A pass is a loop of whole 16-byte vectors, several of them in flight per
// thread at 512 threads an SM; 768 and 1024 threads with fewer in flight each
// read as fast, but the fixed work of a thread (its column's coefficients, sums
// and joins: as many instructions as about 25 vectors) then weighs more (decoder
// size 27.3 us).  Packed fp32 instructions (two lanes an issue slot) carry the
// arithmetic; SiLU's exponential and reciprocal take the special-function pipe
// to 0.49 of its rate at that size and 0.65 at [16, 112x112, 512] fp16.
//
// Statistics: a thread sums x - k and (x - k)^2 with k one of its own values and
// makes its mean and M2 of them, M2 being the sum of squared distances from the
// mean; the threads of a column are joined about one of their means, the columns
// of a group about the group's, blocks about the mean of one.  What an M2 is the
// difference of is never much larger than it, however far the mean is from 0: k is
// the middle() one of four values, so at least two of the thread's n <= 1024 lie
// as far from their mean as k, the sum of (x - k)^2 is at most 1 + n/2 times M2,
// and about 1.5 times where no two of the four are far; likewise for threads and
// blocks.  Measured on [300, 60000, 8] fp16: rstd is off by 5 steps of 2^-24, by
// 8 with a first pixel a thousand deviations off, by 830 where three of the first
// four values of one thread are 10^4 off and no others.  (With one k for a whole
// column, the mean of four of its n <= 2^18 values, it was off by 40000 with the
// first pixel a thousand deviations off.)
#pragma once

#include <string.h>

#include "ct_cuda_util.h"
#include "group_norm.h"
#include "sm100.cuh"
#include "vec16.cuh"

namespace ct {

namespace {

using sm100::cluster_ctarank;
using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

struct Params {      // kernel arguments besides the geometry
    const void *x, *dy, *weight, *bias;
    void *y, *dx, *dweight, *dbias;
    float *mean, *rstd;
    float4 *part;    // forward, per image, slot, chunk and group: (count, mean, M2, -)
    float2 *sums;    // backward, per image, slot, chunk and group: (sum dh, sum dh h)
    float2 *chan;    // backward, per image, chunk, copy and channel: (sum da, sum da h)
    float eps;
    int param_dtype;
    bool vec;
    RngArgs rng;
    int64_t strips;
};

__device__ __forceinline__ float param(const void *p, int c, int dtype, float none) {
    if (!p) return none;
    if (dtype == CT_F32) return ((const float *)p)[c];
    if (dtype == CT_F16) return __half2float(((const __half *)p)[c]);
    return __bfloat162float(((const __nv_bfloat16 *)p)[c]);
}

__device__ __forceinline__ void put_param(void *p, int64_t i, int dtype, float v) {
    if (dtype == CT_F32) ((float *)p)[i] = v;
    else if (dtype == CT_F16) ((__half *)p)[i] = __float2half_rn(v);
    else ((__nv_bfloat16 *)p)[i] = __float2bfloat16_rn(v);
}

// Two neighbours at a time: the packed fp32 instructions of sm_100 do two
// additions, products or multiply-adds per issue slot.
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

__device__ __forceinline__ float2 sigmoid2(float2 a) {
    const float2 e = mul2(a, both(-1.44269504f));
    float2 d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d.x) : "f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d.y) : "f"(e.y));
    d = add2(d, both(1.f));
    float2 s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
    return s;
}

template <int ACT>
__device__ __forceinline__ float2 act_value(float2 a) {
    if (ACT == CT_ACT_RELU) return make_float2(a.x < 0.f ? 0.f : a.x, a.y < 0.f ? 0.f : a.y);
    if (ACT == CT_ACT_SILU) return mul2(a, sigmoid2(a));
    if (ACT == CT_ACT_GELU)
        return make_float2(0.5f * a.x * (1.f + erff(a.x * 0.70710678f)),
                           0.5f * a.y * (1.f + erff(a.y * 0.70710678f)));
    return a;
}

__device__ __forceinline__ float gelu_slope(float a) {
    return 0.5f * (1.f + erff(a * 0.70710678f)) + a * __expf(-0.5f * a * a) * 0.39894228f;
}

template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 a) {
    if (ACT == CT_ACT_RELU) return make_float2(a.x > 0.f ? 1.f : 0.f, a.y > 0.f ? 1.f : 0.f);
    if (ACT == CT_ACT_SILU) {
        const float2 s = sigmoid2(a);
        return fma2(s, fma2(neg2(s), a, a), s);   // s + s a (1 - s)
    }
    if (ACT == CT_ACT_GELU) return make_float2(gelu_slope(a.x), gelu_slope(a.y));
    return both(1.f);
}

// One block's chunk of a strip, and the strip's place: all fields are the
// same in every thread but the last ones.
struct Share {
    int64_t n;             // image
    int tile;              // column tile
    int64_t e0;            // the image's first element
    int head;
    int p0, p1;            // the tile's positions within a row
    int first_group, groups;   // the groups that they meet, counted modulo G
    // this thread's column and row (-1: it has none), its vectors that no end
    // of the image cuts, and those that one cuts
    int col, ty;
    int first, last;                 // whole vectors: rows ty + i * by of the chunk, first <= i < last
    int64_t e, cut_head, cut_tail;   // elements (of i = 0), -1 where there is none
    int64_t r0;                      // the chunk's first row
    int rows;
    int64_t whole_rows;              // the image's vectors that its end does not cut: rows, and those beyond
    int rest;
};

// A block's share of a strip: its chunk is blockIdx.x.  PLAIN:
// a pixel is a whole number of vectors, one column tile, aligned tensors; then
// nothing is cut, a position is its channel and a row a pixel.
template <bool PLAIN>
struct Shares {
    const GnGeom &g;
    const Params &p;
    int tx, ty;

    __device__ __forceinline__ Shares(const GnGeom &geom, const Params &par) : g(geom), p(par) {
        ty = divq(threadIdx.x, g.by_bx);
        tx = threadIdx.x - ty * g.bx;
    }
    __device__ __forceinline__ void get(int64_t strip, Share &t) {
        t.n = strip;
        t.tile = 0;
        if (PLAIN) {
            t.e0 = t.n * g.E;
            t.head = t.p0 = t.first_group = t.first = 0;
            t.p1 = g.C;
            t.groups = g.G;
            t.col = tx;
            t.ty = ty < g.by ? ty : -1;
            t.cut_head = t.cut_tail = -1;
            t.r0 = (int64_t)blockIdx.x * g.rpc;
            t.rows = g.S - t.r0 < g.rpc ? (int)(g.S - t.r0) : g.rpc;   // a cluster may have more blocks than the image rows
            if (t.rows < 0) t.rows = 0;
            t.e = t.e0 + (t.r0 + ty) * g.C + tx * g.V;
            t.last = t.ty >= 0 && t.rows > ty ? divq(t.rows - ty + g.by - 1, g.by_by) : 0;
            t.whole_rows = g.S;
            t.rest = 0;
            return;
        }
        if (g.ctiles > 1) {
            t.n = strip / g.ctiles;
            t.tile = (int)(strip - t.n * g.ctiles);
        }
        t.e0 = t.n * g.E;
        t.head = (int)t.e0 & (g.V - 1);
        t.p0 = t.tile * g.bx * g.V;
        t.p1 = (t.tile + 1) * g.bx < g.LV ? t.p0 + g.bx * g.V : g.LV * g.V;
        if (g.ctiles > 1 && t.p1 > g.copies * g.C)   // the positions after these have no values in any image
            t.p1 = t.p0 < g.copies * g.C ? g.copies * g.C : t.p0;
        const int c = channel(t, t.p0);
        t.first_group = divq(c, g.by_cg);
        t.groups = t.p1 > t.p0 ? divq(t.p1 - t.p0 - 1 + (c - t.first_group * g.Cg), g.by_cg) + 1 : 0;
        if (t.groups > g.G) t.groups = g.G;
        t.col = t.tile * g.bx + tx;
        t.ty = ty < g.by && t.col < g.LV ? ty : -1;
        t.first = t.last = 0;
        t.cut_head = t.cut_tail = -1;
        // the image's vectors that its end does not cut: t.whole_rows rows and t.rest vectors
        t.whole_rows = g.full_rows;
        t.rest = g.full_rest;
        const int over = ((int)g.E & (g.V - 1)) + t.head;
        if (over >= g.V && ++t.rest == g.LV) {
            t.rest = 0;
            ++t.whole_rows;
        }
        t.r0 = (int64_t)blockIdx.x * g.rpc;
        t.rows = g.rows - t.r0 < g.rpc ? (int)(g.rows - t.r0) : g.rpc;
        if (t.rows < 0) t.rows = 0;
        t.e = t.e0 - t.head + g.V * ((t.r0 + ty) * g.LV + t.col);
        if (t.ty < 0) return;
        if (t.head != 0 && t.r0 + ty == 0 && t.col == 0 && t.rows > 0) {
            t.cut_head = t.e;
            t.first = 1;
        }
        const int64_t whole = t.whole_rows + (t.col < t.rest ? 1 : 0) - t.r0;
        const int end = whole < t.rows ? (int)whole : t.rows;
        if (end > ty) t.last = divq(end - ty + g.by - 1, g.by_by);
        if (t.last < t.first) t.last = t.first;
        const int r = ty + t.last * g.by;   // the row after the whole ones
        if ((over & (g.V - 1)) != 0 && r < t.rows && t.r0 + r == t.whole_rows && t.col == t.rest)
            t.cut_tail = t.e + (int64_t)t.last * g.V * g.LV * g.by;
    }
    // the channel at position `pos` of a row
    __device__ __forceinline__ int channel(const Share &t, int pos) const {
        if (PLAIN || g.wraps == 1) return pos;
        const int c = (pos - t.head) % g.C;
        return c < 0 ? c + g.C : c;
    }
};

// Of the tiles below `upto`, how many hold channels of group gi in an image
// whose channels start at position `head` of its rows (tiles run up, so the
// runs of a group's channels, one to a copy, meet theirs in order).
__device__ __forceinline__ int tiles_of(const GnGeom &g, int head, int gi, int upto) {
    const int end = g.copies * g.C;
    int n = 0, next = 0;
    for (int a = gi * g.Cg + head - (g.wraps > 1 ? g.C : 0); a < end; a += g.C) {
        const int lo = max(a, 0), hi = min(a + g.Cg, end) - 1;
        if (hi < lo) continue;
        const int last = divq(hi, g.by_tile);
        n += max(0, min(last + 1, upto) - max(divq(lo, g.by_tile), next));
        next = last + 1;
    }
    return n;
}

// The image's first slots in the workspace, and group gi's from this block's
// chunk there on.
template <bool PLAIN>
__device__ __forceinline__ int64_t slots_of(const GnGeom &g, const Share &t) {
    return (PLAIN ? t.n : t.n * g.slots) * g.chunks;
}
template <bool PLAIN>
__device__ __forceinline__ int64_t slot_at(const GnGeom &g, const Share &t, int gi) {
    return PLAIN || g.ctiles == 1 ? gi : (int64_t)tiles_of(g, t.head, gi, t.tile) * g.chunks * g.G + gi;
}

// The elements of a cut vector that are the image's.
__device__ __forceinline__ uint32_t cut_bits(const GnGeom &g, const Share &t, int64_t e) {
    uint32_t m = 0;
    for (int k = 0; k < g.V; ++k)
        if (e + k >= t.e0 && e + k < t.e0 + g.E) m |= 1u << k;
    return m;
}

__device__ __forceinline__ float &lane_of(float2 &v, int k) { return k & 1 ? v.y : v.x; }

// The cluster's barrier in two halves. The aligned forms want their warp
// together, which a branch or a loop by lane just before does not promise.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Nothing {
    template <typename Get>
    __device__ __forceinline__ void operator()(int, Get) const {}
};

// f(element, pairs of each of N tensors, bits) for a thread's vectors: the
// whole ones with U in flight, then those that an end of the image cuts (the
// elements outside `bits` read as 0); on unaligned tensors all one by one.
// pre(n, get) runs before the first of them, while the first loads are in
// flight: n whole vectors follow, get(i) is number i < min(n, U) of the first
// tensor's.
template <typename T, bool PLAIN, int N, int U, typename Pre, typename F>
__device__ __forceinline__ void stream(const GnGeom &g, const Share &t, const T *const (&src)[N], bool vec, Pre pre,
                                       F f) {
    constexpr int V = kVec<T>, P = V / 2;
    const int64_t step = (int64_t)V * g.LV * g.by;
    if (PLAIN || vec) {
        int left = t.last - (PLAIN ? 0 : t.first);
        int64_t e = t.e + (PLAIN ? 0 : t.first) * step;
        uint4 w[U][N];
        auto load = [&](int u, int64_t at) {
#pragma unroll
            for (int j = 0; j < N; ++j) w[u][j] = __ldg(reinterpret_cast<const uint4 *>(src[j] + at));
        };
        auto use = [&](int u) {
            float2 v[N][P];
#pragma unroll
            for (int j = 0; j < N; ++j) unpack(w[u][j], v[j], T());
            f(e + u * step, v, ~0u);
        };
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < left) load(u, e + u * step);
        pre(left, [&](int i) { return w[i][0]; });
        // the next ones are loaded together, forward in two halves so that some
        // are always on their way (decoder size 25.4 us, 26.6 all together; one by
        // one as registers free took 254 at vocoder size in place of 150)
        constexpr int H = N == 1 ? (U + 1) / 2 : U;
        while (left > 0) {
#pragma unroll
            for (int h = 0; h < U; h += H) {
#pragma unroll
                for (int u = h; u < h + H && u < U; ++u)
                    if (u < left) use(u);
#pragma unroll
                for (int u = h; u < h + H && u < U; ++u)
                    if (u + U < left) load(u, e + (u + U) * step);
            }
            e += U * step;
            left -= U;
        }
        if (PLAIN || (t.cut_head < 0 && t.cut_tail < 0)) return;
    } else {
        pre(t.last - t.first, [&](int i) { return gather(src[0] + t.e + (t.first + i) * step); });
    }
#pragma unroll 1
    for (int i = vec ? t.last : t.first; i < t.last + 2; ++i) {
        const int64_t e = i < t.last ? t.e + i * step : i == t.last ? t.cut_head : t.cut_tail;
        if (e < 0) continue;
        const uint32_t bits = i < t.last ? ~0u : cut_bits(g, t, e);
        float2 v[N][P];
#pragma unroll
        for (int j = 0; j < N; ++j) load_some(src[j] + e, bits, v[j]);
        f(e, v, bits);
    }
}

__device__ __forceinline__ float at_least_0(float v) { return v < 0.f ? 0.f : v; }   // NaN stays

__device__ __forceinline__ float group_sum(float v, int lanes) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2)
        if (o < lanes) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// log2 of the lanes that share one of `n` things: a power of two up to 32.
__device__ __forceinline__ int log_lanes_for(int n) {
    return n >= kThreads ? 0 : min(5, 31 - __clz(kThreads / n));
}

// log2 of the warps that share one of `n` groups: a block's eight among fewer
// than eight groups.  The general kernels only ([8, 16383, 127] fp16 in one
// group 29.7 us in place of 31.9): the plain ones have short sums, and sharing
// costs them about 1% at most sizes (decoder size 25.6 us in place of 25.3,
// backward [16, 112x112, 512] fp16 187.5 in place of 187.0) where shapes of one
// group and few pixels would gain ([8, 256, 2048] bf16 18.8 in place of 24.5).
__device__ __forceinline__ int log_warps_for(int n) { return n == 1 ? 3 : n == 2 ? 2 : n <= 4 ? 1 : 0; }

__device__ __forceinline__ int wrap_group(const GnGeom &g, int gi) { return gi >= g.G ? gi - g.G : gi; }

// Store to shared address `p` of the cluster's block `rank`.
__device__ __forceinline__ void push(float4 *p, int rank, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                     sm100::mapa_shared(sm100::smem_u32(p), rank)),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// A thread's V values of a per-position array.
template <int V>
__device__ __forceinline__ void own(const float *at, const Share &t, float2 (&v)[V / 2]) {
    const float4 *q = reinterpret_cast<const float4 *>(at + (t.col * V - t.p0));
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
        const float4 w = q[j];
        v[2 * j] = make_float2(w.x, w.y);
        v[2 * j + 1] = make_float2(w.z, w.w);
    }
}
template <int V>
__device__ __forceinline__ void put_own(float *at, const float2 (&v)[V / 2]) {
    float4 *q = reinterpret_cast<float4 *>(at + threadIdx.x * V);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) q[j] = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
}

// f(position in the tile, channel, group, the tile's number of the group)
template <bool PLAIN, typename F>
__device__ __forceinline__ void each_position(const GnGeom &g, const Shares<PLAIN> &shares, const Share &t, F f) {
    for (int pos = threadIdx.x; pos < t.p1 - t.p0; pos += kThreads) {
        if (PLAIN) {
            const int gi = divq(pos, g.by_cg);
            f(pos, pos, gi, gi);
            continue;
        }
        const int c = shares.channel(t, t.p0 + pos), gi = divq(c, g.by_cg);
        f(pos, c, gi, gi >= t.first_group ? gi - t.first_group : gi - t.first_group + g.G);
    }
}

// f(position in the tile) for lane `lane` of `lanes` over the positions of a
// group (or, with count 1, of a channel): channels c .. c + count - 1.
template <bool PLAIN, typename F>
__device__ __forceinline__ void group_positions(const GnGeom &g, const Share &t, int c, int count, int lane, int lanes,
                                                F f) {
    if (!PLAIN && g.ctiles > 1) {   // run by run: the tile may hold few of the group's channels
        for (int a = c + t.head - t.p0 - (g.wraps > 1 ? g.C : 0); a < t.p1 - t.p0; a += g.C)
            for (int pos = max(a, 0) + lane; pos < min(a + count, t.p1 - t.p0); pos += lanes) f(pos);
        return;
    }
    for (int j = lane; j < count; j += lanes) {
        if (PLAIN) {
            f(c + j);
            continue;
        }
        int pos = c + j + t.head;
        while (pos >= g.C) pos -= g.C;   // more than once where C is below the head
        for (; pos < t.p1; pos += g.C) f(pos);
    }
}

// ---- forward ----------------------------------------------------------------

// Dynamic shared memory of the forward kernels.
struct FwdShared {
    float *nmean, *mul, *add;   // per position of the tile: a = (x + nmean) mul + add; nmean before that
                                // what the columns' sums are about
    float *sums;                // the threads' means, M2 and counts, then their columns' sums
    float4 *pushed;             // [2][cluster][groups]: the cluster's (count, mean, M2), taking turns by strip
    float2 *stat;               // (mean, rstd) of the groups
    int groups;
    __device__ __forceinline__ FwdShared(const GnGeom &g) {
        extern __shared__ float4 dynamic[];
        const int width = g.bx * g.V;
        groups = groups_max(g);
        nmean = (float *)dynamic;
        mul = nmean + width;
        add = mul + width;
        sums = add + width;
        pushed = (float4 *)(sums + kThreads * g.V * (g.wraps > 1 ? 3 : 2));
        stat = (float2 *)(pushed + 2 * g.cluster * groups);
    }
};
size_t forward_smem(const GnGeom &g) {
    return (size_t)g.bx * g.V * 12 + (size_t)kThreads * g.V * (g.wraps > 1 ? 12 : 8) +
           (size_t)groups_max(g) * (32 * g.cluster + 8);
}

// The larger of the smaller ones of two pairs: at least two of the four lie on
// either side of it (itself among them), so that it is as far from their mean as
// two of them, and no single far one is taken.
__device__ __forceinline__ float middle(float a, float b, float c, float d) { return fmaxf(fminf(a, b), fminf(c, d)); }

// Per position, runs of thread rows apart: the sums of n (m - r) and of
// M2 + n (m - r)^2 about r = sh.nmean, and of n where rows are not whole.
struct ColumnStats {
    const float *s, *q, *n;
    int width, segs;
    __device__ __forceinline__ float sum(const float *at) const {
        float v = at[0];
        for (int i = 1; i < segs; ++i) v += at[i * width];
        return v;
    }
};

// The thread rows of sh.sums (m, M2 and n of each) joined, about the middle one
// of four rows' means. Row y of an array is read by one thread only but for the
// means', so the sums go to the first rows of M2.
__device__ __forceinline__ ColumnStats column_stats(const GnGeom &g, const Share &t, const FwdShared &sh, bool counted) {
    const int width = g.bx * g.V, apart = kThreads * g.V;
    float *means = sh.sums, *m2 = means + apart, *counts = m2 + apart;
    int segs = 1;
    while (segs * 2 * width <= kThreads && segs * 4 <= g.by) segs *= 2;
    __syncthreads();
    if (g.by == 1) return {means, m2, counts, width, 1};   // the row's own, with s = 0
    const int runs = segs * width, all = g.by * width, rounds = divq(t.rows, g.by_by);
    const int more = (t.rows - rounds * g.by) * width;   // rows below have a value more
    const float least = (float)rounds, most = (float)(rounds + 1);
    const int last = max(min(g.by, t.rows) - 1, 0);   // the last row that has values
    for (int i = threadIdx.x; i < runs; i += kThreads) {
        int pos = i;
        while (pos >= width) pos -= width;
        const float r = middle(means[pos], means[pos + min(1, last) * width], means[pos + min(2, last) * width],
                               means[pos + min(3, last) * width]);
        float n = 0.f, s = 0.f, q = 0.f;
#pragma unroll 8
        for (int y = i; y < all; y += runs) {
            const float ny = counted ? counts[y] : y - pos < more ? most : least;
            const float d = means[y] - r, w = ny * d;
            n += ny;
            s += w;
            q += m2[y] + w * d;
        }
        if (i == pos) sh.nmean[pos] = r;
        m2[i] = s;
        m2[runs + i] = q;
        if (counted) counts[i] = n;
    }
    __syncthreads();
    return {m2, m2 + runs, counts, width, segs};
}

// The shift k of a thread's channels, of its n whole vectors get(i): the middle()
// of the first four's values, or where there is no whole vector the image's first
// pixel. One of the values, so that x - k has x's low bits, which vary: with bits
// of k below x's steps, the same in every term, each addition rounds the same way
// once a sum has grown past them (rstd of 60000 fp16 values was off by 50 steps
// of 2^-24).
template <typename T, bool PLAIN, typename Get>
__device__ __forceinline__ void shift(const GnGeom &g, const Params &p, const Shares<PLAIN> &shares, const Share &t,
                                      int n, Get get, float2 (&k)[kVec<T> / 2]) {
    constexpr int V = kVec<T>, P = V / 2;
#pragma unroll
    for (int j = 0; j < P; ++j) k[j] = both(0.f);
    if (n > 0) {
        const uint4 a = get(0), b = n > 1 ? get(1) : a, c = n > 2 ? get(2) : b, d = n > 3 ? get(3) : c;
        unpack(larger(smaller(a, b, T()), smaller(c, d, T()), T()), k, T());
    } else if (!PLAIN) {
        int c = shares.channel(t, V * t.col);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            lane_of(k[i / 2], i) = to_f<T>(((const T *)p.x)[t.e0 + c]);
            if (++c == g.C) c = 0;
        }
    }
}

// The running join of (count, mean, M2) triples about a reference r, the mean
// of one of them: sum n (m - r) and sum M2 + n (m - r)^2.  As r is the mean of
// part of the values, the distance that the second carries is at most their M2
// times the number of parts of that size (of half of it where r is a middle()).
struct Joined {
    float n, s, q, r;
    __device__ __forceinline__ void add(float4 v) {
        if (v.x > 0.f) {
            const float d = v.y - r, w = v.x * d;
            n += v.x;
            s += w;
            q += v.z + w * d;
        }
    }
    __device__ __forceinline__ float4 triple() const {
        const float m = n > 0.f ? s / n : 0.f;
        return make_float4(n, r + m, at_least_0(q - s * m), 0.f);
    }
};

// This block's statistics: ready(), then emit(group of the tile, lane, lanes,
// triple) for each group, its lanes together.
template <typename T, bool PLAIN, typename Ready, typename Emit>
__device__ __forceinline__ void block_stats(const GnGeom &g, const Params &p, const Shares<PLAIN> &shares, const Share &t,
                                            const FwdShared &sh, Ready ready, Emit emit) {
    constexpr int V = kVec<T>, P = V / 2;
    {
        float2 nk[P], s[P], q[P];
        float n[V];
#pragma unroll
        for (int j = 0; j < P; ++j) s[j] = q[j] = both(0.f);
        const float whole = (float)(t.last - t.first);
#pragma unroll
        for (int k = 0; k < V; ++k) n[k] = whole;
        const T *const x[1] = {(const T *)p.x};
        auto pre = [&](int whole_ones, auto get) {
            shift<T, PLAIN>(g, p, shares, t, whole_ones, get, nk);
#pragma unroll
            for (int j = 0; j < P; ++j) nk[j] = neg2(nk[j]);
        };
        if (t.ty >= 0)
            stream<T, PLAIN, 1, kForwardUnroll>(g, t, x, p.vec, pre, [&](int64_t, const float2 (&v)[1][P], uint32_t bits) {
            if (bits == ~0u) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 d = add2(v[0][j], nk[j]);
                    s[j] = add2(s[j], d);
                    q[j] = fma2(d, d, q[j]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if ((bits >> k) & 1u) {
                        const float d = (k & 1 ? v[0][k / 2].y : v[0][k / 2].x) + lane_of(nk[k / 2], k);
                        lane_of(s[k / 2], k) += d;
                        lane_of(q[k / 2], k) += d * d;
                        n[k] += 1.f;
                    }
            }
        });
        if (t.ty >= 0) {   // to mean and M2
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 inv = make_float2(n[2 * j] > 0.f ? __fdividef(1.f, n[2 * j]) : 0.f,
                                               n[2 * j + 1] > 0.f ? __fdividef(1.f, n[2 * j + 1]) : 0.f);
                const float2 d = mul2(s[j], inv);
                q[j] = fma2(neg2(s[j]), d, q[j]);
                q[j] = make_float2(at_least_0(q[j].x), at_least_0(q[j].y));
                s[j] = add2(d, neg2(nk[j]));
            }
            if (g.by == 1) {   // nothing to join: about its own mean
                put_own<V>(sh.nmean, s);
#pragma unroll
                for (int j = 0; j < P; ++j) s[j] = both(0.f);
            }
            put_own<V>(sh.sums, s);
            put_own<V>(sh.sums + kThreads * V, q);
            if (!PLAIN && g.wraps > 1) {
                float2 c[P];
#pragma unroll
                for (int j = 0; j < P; ++j) c[j] = make_float2(n[2 * j], n[2 * j + 1]);
                put_own<V>(sh.sums + 2 * kThreads * V, c);
            }
        }
    }
    const bool counted = !PLAIN && g.wraps > 1;   // counts differ by position
    const ColumnStats cols = column_stats(g, t, sh, counted);
    // per group: its positions' means, then the distances from their mean
    const int log = log_lanes_for(t.groups), lanes = 1 << log, lane = threadIdx.x & (lanes - 1);
    const int logw = PLAIN ? 0 : log_warps_for(t.groups), warps = 1 << logw;
    __shared__ float4 shares_of_warps[kThreads / 32];
    ready();
    const float rows = (float)t.rows, by_rows = t.rows > 0 ? __fdividef(1.f, rows) : 0.f;
    for (int gb = 0; gb < t.groups; gb += kThreads >> (log + logw)) {
        const int lg = gb + (threadIdx.x >> (log + logw)), at = threadIdx.x & ((lanes << logw) - 1);
        const int c = wrap_group(g, t.first_group + lg) * g.Cg, many = lg < t.groups ? g.Cg : 0;
        float sn = 0.f, sm = 0.f, sq = 0.f;
        group_positions<PLAIN>(g, t, c, many, at, lanes << logw, [&](int pos) {
            const float n = counted ? cols.sum(cols.n + pos) : rows;
            sn += n;
            sm += n * sh.nmean[pos] + cols.sum(cols.s + pos);
        });
        sn = group_sum(sn, lanes);
        sm = group_sum(sm, lanes);
        const float m = sn > 0.f ? __fdividef(sm, sn) : 0.f;
        group_positions<PLAIN>(g, t, c, many, at, lanes << logw, [&](int pos) {
            const float n = counted ? cols.sum(cols.n + pos) : rows;
            const float inv = counted ? (n > 0.f ? __fdividef(1.f, n) : 0.f) : by_rows;
            const float s = cols.sum(cols.s + pos), d = sh.nmean[pos] + s * inv - m;
            sq += at_least_0(cols.sum(cols.q + pos) - s * s * inv) + n * d * d;
        });
        sq = group_sum(sq, lanes);
        float4 v = make_float4(sn, m, sq, 0.f);
        if (logw > 0) {   // one step: the warps' triples joined
            if (lane == 0) shares_of_warps[threadIdx.x / 32] = v;
            __syncthreads();
            Joined all = {0.f, 0.f, 0.f, 0.f};
            if (at < 32)
                for (int i = 0; i < warps; ++i) {
                    v = shares_of_warps[threadIdx.x / 32 + i];
                    if (all.n == 0.f) all.r = v.y;
                    all.add(v);
                }
            v = all.triple();
        }
        if (lg < t.groups && at < lanes) emit(lg, lane, lanes, v);
    }
}

// The triples that the cluster's blocks pushed, joined: one thread per group.
__device__ __forceinline__ float4 join_pushed(const FwdShared &sh, const float4 *pushed, int cluster, int lg) {
    Joined j = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < cluster; ++i) {
        const float4 v = pushed[i * sh.groups + lg];
        if (j.n == 0.f) j.r = v.y;
        j.add(v);
    }
    return j.triple();
}

// (mean, rstd) of a group from its joined sums, kept and written.
__device__ __forceinline__ void put_stat(const GnGeom &g, const Params &p, const Share &t, const FwdShared &sh, int lg,
                                         float4 v) {
    const float rstd = 1.f / sqrtf(__fdividef(v.z, fmaxf(v.x, 1.f)) + p.eps);
    sh.stat[lg] = make_float2(v.y, rstd);
    if (blockIdx.x == 0) {   // tiles that share a group write the same
        const int64_t at = t.n * g.G + wrap_group(g, t.first_group + lg);
        if (p.mean) p.mean[at] = v.y;
        if (p.rstd) p.rstd[at] = rstd;
    }
}

// The parameters of the tile's positions, before their statistics are known.
template <bool PLAIN>
__device__ __forceinline__ void stage_params(const GnGeom &g, const Params &p, const Shares<PLAIN> &shares, const Share &t,
                                             const FwdShared &sh) {
    each_position(g, shares, t, [&](int pos, int c, int, int) {
        sh.mul[pos] = param(p.weight, c, p.param_dtype, 1.f);
        sh.add[pos] = param(p.bias, c, p.param_dtype, 0.f);
    });
}

// y of this block's rows from sh.stat.
template <typename T, bool PLAIN, int ACT, int DROP>
__device__ __forceinline__ void apply_rows(const GnGeom &g, const Params &p, const Shares<PLAIN> &shares, const Share &t,
                                           const FwdShared &sh, const Philox<DROP == 1> &philox) {
    constexpr int V = kVec<T>, P = V / 2;
    __syncthreads();
    each_position(g, shares, t, [&](int pos, int, int, int lg) {
        const float2 s = sh.stat[lg];
        sh.nmean[pos] = -s.x;
        sh.mul[pos] *= s.y;
    });
    __syncthreads();
    float2 nmean[P], mul[P], add[P];
    own<V>(sh.nmean, t, nmean);
    own<V>(sh.mul, t, mul);
    own<V>(sh.add, t, add);
    const T *const x[1] = {(const T *)p.x};
    T *y = (T *)p.y;
    const uint32_t limit = drop_limit(p.rng.threshold);
    constexpr bool on = DROP != 0;
    if (t.ty >= 0)
        stream<T, PLAIN, 1, kForwardUnroll>(g, t, x, p.vec, Nothing(), [&](int64_t e, float2 (&v)[1][P], uint32_t bits) {
        uint32_t w[P];
        if (on) draw(philox, (uint64_t)e, w);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            v[0][j] = act_value<ACT>(fma2(add2(v[0][j], nmean[j]), mul[j], add[j]));
            if (on) v[0][j] = drop_pair(w[j], limit, p.rng.scale, v[0][j]);
        }
        if (PLAIN) store_vec(y + e, true, v[0]);
        else if (bits == ~0u) store_vec(y + e, p.vec, v[0]);
        else store_some(y + e, bits, v[0]);
    });
    __syncthreads();
}

template <typename T, bool PLAIN, int ACT, int DROP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    gn_fused_kernel(const __grid_constant__ GnGeom g, const __grid_constant__ Params p) {
    const FwdShared sh(g);
    Shares<PLAIN> shares(g, p);
    Share t;
    int turn = 0;
    cluster_arrive();   // every block of the cluster runs before any stores to it: its push waits
    const int rank = cluster_ctarank();
    const Philox<DROP == 1> philox(p.rng);
    for (int64_t s = blockIdx.y; s < p.strips; s += gridDim.y) {
        shares.get(s, t);
        float4 *pushed = sh.pushed + turn * g.cluster * sh.groups;
        turn ^= 1;
        stage_params(g, p, shares, t, sh);
        block_stats<T, PLAIN>(
            g, p, shares, t, sh,
            [&] {
                if (s == blockIdx.y) cluster_wait();
            },
            [&](int lg, int lane, int lanes, float4 v) {
                for (int i = lane; i < g.cluster; i += lanes) push(pushed + rank * sh.groups + lg, i, v);
            });
        cluster_arrive();
        cluster_wait();
        for (int lg = threadIdx.x; lg < t.groups; lg += kThreads)
            put_stat(g, p, t, sh, lg, join_pushed(sh, pushed, g.cluster, lg));
        apply_rows<T, PLAIN, ACT, DROP>(g, p, shares, t, sh, philox);
    }
}

template <typename T, bool PLAIN>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    gn_stats_kernel(const __grid_constant__ GnGeom g, const __grid_constant__ Params p) {
    const FwdShared sh(g);
    griddep_launch_dependents();
    Shares<PLAIN> shares(g, p);
    Share t;
    for (int64_t s = blockIdx.y; s < p.strips; s += gridDim.y) {
        shares.get(s, t);
        float4 *out = p.part + (slots_of<PLAIN>(g, t) + blockIdx.x) * g.G;
        block_stats<T, PLAIN>(
            g, p, shares, t, sh, [] {},
            [&](int lg, int lane, int, float4 v) {
                if (lane == 0) out[slot_at<PLAIN>(g, t, wrap_group(g, t.first_group + lg))] = v;
            });
        __syncthreads();
    }
}

// A group's parts, which follow each other in the workspace, G apart.
template <bool PLAIN>
__device__ __forceinline__ int parts_of(const GnGeom &g, const Share &t, int gi) {
    return (PLAIN || g.ctiles == 1 ? 1 : tiles_of(g, t.head, gi, g.ctiles)) * g.chunks;
}

// f(group of the tile, triple) with an image's parts joined: a thread takes
// every `slices`-th part of a group, neighbours neighbouring groups. The slices
// are as many in every tile, so that the tiles which share a group add its
// parts in the same order and find the same bits.
template <bool PLAIN, typename F>
__device__ __forceinline__ void join_parts(const GnGeom &g, const Share &t, const FwdShared &sh, const float4 *part,
                                           F f) {
    const float4 *in = part + slots_of<PLAIN>(g, t) * g.G;
    float *acc = sh.sums;   // three arrays of kThreads
    const int log = log_lanes_for(g.tile_groups);   // at most 32 slices
    for (int gb = 0; gb < t.groups; gb += kThreads >> log) {
        const int here = t.groups - gb < kThreads >> log ? t.groups - gb : kThreads >> log;   // groups of this step
        const int slices = 1 << log, slice = threadIdx.x / here, lg = gb + threadIdx.x - slice * here;
        Joined j = {0.f, 0.f, 0.f, 0.f};
        if (slice < slices) {
            const int gi = wrap_group(g, t.first_group + lg);
            const float4 *q = in + gi;
            const int parts = parts_of<PLAIN>(g, t, gi);
            // about the middle() of four parts of the tile that the group's first channel is in, of which
            // the first surely has values
            const int first = PLAIN || g.ctiles == 1
                                  ? 0
                                  : tiles_of(g, t.head, gi, divq(gi * g.Cg + t.head, g.by_tile)) * g.chunks;
            float4 some[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) some[k] = q[(int64_t)(first + (int)((int64_t)g.chunks * k / 4)) * g.G];
#pragma unroll
            for (int k = 1; k < 4; ++k)
                if (some[k].x == 0.f) some[k].y = some[0].y;
            j.r = middle(some[0].y, some[1].y, some[2].y, some[3].y);
#pragma unroll 8
            for (int i = slice; i < parts; i += slices) j.add(q[(int64_t)i * g.G]);
            acc[threadIdx.x] = j.n;
            acc[kThreads + threadIdx.x] = j.s;
            acc[2 * kThreads + threadIdx.x] = j.q;
        }
        __syncthreads();
        if (threadIdx.x < here) {
            Joined a = j;
            for (int i = 1; i < slices; ++i) {
                a.n += acc[i * here + threadIdx.x];
                a.s += acc[kThreads + i * here + threadIdx.x];
                a.q += acc[2 * kThreads + i * here + threadIdx.x];
            }
            f(lg, a.triple());
        }
        __syncthreads();
    }
}

template <typename T, bool PLAIN, int ACT, int DROP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    gn_apply_kernel(const __grid_constant__ GnGeom g, const __grid_constant__ Params p) {
    const FwdShared sh(g);
    griddep_launch_dependents();
    Shares<PLAIN> shares(g, p);
    Share t;
    const Philox<DROP == 1> philox(p.rng);
    bool waited = false;
    for (int64_t s = blockIdx.y; s < p.strips; s += gridDim.y) {
        shares.get(s, t);
        stage_params(g, p, shares, t, sh);
        if (!waited) griddep_wait();
        waited = true;
        join_parts<PLAIN>(g, t, sh, p.part, [&](int lg, float4 v) { put_stat(g, p, t, sh, lg, v); });
        apply_rows<T, PLAIN, ACT, DROP>(g, p, shares, t, sh, philox);
    }
    if (!waited) griddep_wait();
}

// ---- backward ---------------------------------------------------------------

// Dynamic shared memory of the backward kernels.
struct BwdShared {
    float *nmean, *mul, *add;   // per position of the tile: a = (x + nmean) mul + add
    float *weight, *rstd;       // per position
    float *sums;                // the threads' sums of da and of da (x - mean); row 0 the block's per position
    float4 *pushed;             // [2][cluster][groups]: the cluster's (sum dh, sum dh h), taking turns by strip
    float2 *stat;               // the groups' means of both
    int groups;
    __device__ __forceinline__ BwdShared(const GnGeom &g) {
        extern __shared__ float4 dynamic[];
        const int width = g.bx * g.V;
        groups = groups_max(g);
        nmean = (float *)dynamic;
        mul = nmean + width;
        add = mul + width;
        weight = add + width;
        rstd = weight + width;
        sums = rstd + width;
        pushed = (float4 *)(sums + kThreads * g.V * 2);
        stat = (float2 *)(pushed + 2 * g.cluster * groups);
    }
};
size_t backward_smem(const GnGeom &g) {
    return (size_t)g.bx * g.V * 20 + (size_t)kThreads * g.V * 8 + (size_t)groups_max(g) * (32 * g.cluster + 8);
}

// Sums over the thread rows of the two arrays [by][bx * V], kThreads * V apart,
// of sh.sums: an array's rows are cut into a few runs, run s is summed into row
// s, and at(k, pos) adds the runs of array k.
struct Columns {
    const float *sums;
    int width, apart, segs;
    __device__ __forceinline__ float at(int k, int pos) const {
        const float *a = sums + k * apart + pos;
        float v = a[0];
        for (int s = 1; s < segs; ++s) v += a[s * width];
        return v;
    }
};
__device__ __forceinline__ Columns column_sums(const GnGeom &g, float *sums) {
    Columns c = {sums, g.bx * g.V, kThreads * g.V, 1};
    while (c.segs * 4 * c.width <= kThreads && c.segs * 4 <= g.by) c.segs *= 2;
    __syncthreads();
    const int runs = c.segs * c.width;   // of an array; consecutive threads take consecutive positions
    if (g.by > 1)
        for (int i = threadIdx.x; i < 2 * runs; i += kThreads) {
            const int k = i >= runs ? 1 : 0, j = i - k * runs;
            float *a = sums + k * c.apart + j;   // row s, position pos of run s: this thread's own
            const int rows = g.by * c.width - j;
            float v = 0.f;
#pragma unroll 8
            for (int y = 0; y < rows; y += runs) v += a[y];
            a[0] = v;
        }
    __syncthreads();
    return c;
}

// The coefficients of the tile's positions, and this thread's.
template <int V>
struct Coef {
    float2 nmean[V / 2], mul[V / 2], add[V / 2];
    template <bool PLAIN>
    __device__ __forceinline__ Coef(const GnGeom &g, const Params &p, const Shares<PLAIN> &shares, const Share &t,
                                    const BwdShared &sh) {
        const float *mean = p.mean + t.n * g.G, *rstd = p.rstd + t.n * g.G;
        each_position(g, shares, t, [&](int pos, int c, int gi, int) {
            const float w = param(p.weight, c, p.param_dtype, 1.f), r = rstd[gi];
            sh.nmean[pos] = -mean[gi];
            sh.mul[pos] = r * w;
            sh.add[pos] = param(p.bias, c, p.param_dtype, 0.f);
            sh.weight[pos] = w;
            sh.rstd[pos] = r;
        });
        __syncthreads();
        own<V>(sh.nmean, t, nmean);
        own<V>(sh.mul, t, mul);
        own<V>(sh.add, t, add);
    }
};

// da of a pair; v becomes x - mean
template <int ACT>
__device__ __forceinline__ float2 grad_a(float2 &v, float2 d, float2 nmean, float2 mul, float2 add, bool on,
                                         uint32_t word, uint32_t limit, float scale) {
    v = add2(v, nmean);
    if (on) d = drop_pair(word, limit, scale, d);
    if (ACT == CT_ACT_IDENTITY) return d;
    return mul2(d, act_slope<ACT>(fma2(v, mul, add)));
}

// This block's sums: per channel to p.chan; ready(), then emit(group of the
// tile, lane, lanes, sums) for each group, its lanes together.
template <typename T, bool PLAIN, int ACT, int DROP, typename Ready, typename Emit>
__device__ __forceinline__ void block_sums(const GnGeom &g, const Params &p, const Share &t, const Coef<kVec<T>> &f,
                                           const BwdShared &sh, const Philox<DROP == 1> &philox, Ready ready, Emit emit) {
    constexpr int V = kVec<T>, P = V / 2;
    {
        const uint32_t limit = drop_limit(p.rng.threshold);
        constexpr bool on = DROP != 0;
        float2 u[P], w[P];
#pragma unroll
        for (int j = 0; j < P; ++j) u[j] = w[j] = both(0.f);
        const T *const src[2] = {(const T *)p.x, (const T *)p.dy};
        if (t.ty >= 0)
            stream<T, PLAIN, 2, DROP || !PLAIN ? kFewerUnroll : kBackwardUnroll>(g, t, src, p.vec, Nothing(), [&](int64_t e, float2 (&v)[2][P], uint32_t bits) {
            uint32_t r[P];
            if (on) draw(philox, (uint64_t)e, r);
            if (bits != ~0u) {   // outside the image x is the mean and dy is 0: nothing is added
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (!((bits >> (2 * j)) & 1u)) v[0][j].x = -f.nmean[j].x;
                    if (!((bits >> (2 * j + 1)) & 1u)) v[0][j].y = -f.nmean[j].y;
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 da = grad_a<ACT>(v[0][j], v[1][j], f.nmean[j], f.mul[j], f.add[j], on, on ? r[j] : 0,
                                               limit, p.rng.scale);
                u[j] = add2(u[j], da);
                w[j] = fma2(da, v[0][j], w[j]);
            }
        });
        if (t.ty >= 0) {
            put_own<V>(sh.sums, u);
            put_own<V>(sh.sums + kThreads * V, w);
        }
    }
    const Columns cols = column_sums(g, sh.sums);
    if (p.chan) {
        float2 *out = p.chan + (t.n * g.chunks + blockIdx.x) * g.copies * g.C;
        if (!PLAIN && g.ctiles > 1) {   // the tile's own, copies apart
            for (int pos = threadIdx.x; pos < t.p1 - t.p0; pos += kThreads)
                out[t.p0 + pos] = make_float2(cols.at(0, pos), cols.at(1, pos) * sh.rstd[pos]);
        } else {
            for (int c = threadIdx.x; c < g.C; c += kThreads) {
                float2 s = both(0.f);
                group_positions<PLAIN>(g, t, c, 1, 0, 1, [&](int pos) {
                    s = add2(s, make_float2(cols.at(0, pos), cols.at(1, pos) * sh.rstd[pos]));
                });
                out[c] = s;
            }
        }
    }
    const int log = log_lanes_for(t.groups), lanes = 1 << log, lane = threadIdx.x & (lanes - 1);
    const int logw = PLAIN ? 0 : log_warps_for(t.groups), warps = 1 << logw;
    __shared__ float2 shares_of_warps[kThreads / 32];
    ready();
    for (int gb = 0; gb < t.groups; gb += kThreads >> (log + logw)) {
        const int lg = gb + (threadIdx.x >> (log + logw)), at = threadIdx.x & ((lanes << logw) - 1);
        float2 s = both(0.f);
        group_positions<PLAIN>(g, t, wrap_group(g, t.first_group + lg) * g.Cg, lg < t.groups ? g.Cg : 0, at, lanes << logw,
                               [&](int pos) {
                                   const float w = sh.weight[pos];
                                   s = add2(s, make_float2(w * cols.at(0, pos), w * sh.rstd[pos] * cols.at(1, pos)));
                               });
        s.x = group_sum(s.x, lanes);
        s.y = group_sum(s.y, lanes);
        if (logw > 0) {   // one step: the warps' sums joined
            if (lane == 0) shares_of_warps[threadIdx.x / 32] = s;
            __syncthreads();
            if (at < 32)
                for (int i = 1; i < warps; ++i) s = add2(s, shares_of_warps[threadIdx.x / 32 + i]);
        }
        if (lg < t.groups && at < lanes) emit(lg, lane, lanes, s);
    }
}

__device__ __forceinline__ float2 join_pushed(const BwdShared &sh, const float4 *pushed, int cluster, int lg) {
    float2 s = both(0.f);
    for (int i = 0; i < cluster; ++i) {
        const float4 v = pushed[i * sh.groups + lg];
        s = add2(s, make_float2(v.x, v.y));
    }
    return s;
}

// dx of this block's rows from sh.stat.
template <typename T, bool PLAIN, int ACT, int DROP>
__device__ __forceinline__ void grad_rows(const GnGeom &g, const Params &p, const Shares<PLAIN> &shares, const Share &t,
                                          const Coef<kVec<T>> &f, const BwdShared &sh, const Philox<DROP == 1> &philox) {
    constexpr int V = kVec<T>, P = V / 2;
    __syncthreads();
    float *m0 = sh.sums, *m1 = sh.sums + g.bx * V;   // per position: -rstd mean(dh), -rstd^2 mean(dh h)
    each_position(g, shares, t, [&](int pos, int, int, int lg) {
        const float2 s = sh.stat[lg];
        const float r = sh.rstd[pos];
        m0[pos] = -r * s.x;
        m1[pos] = -r * r * s.y;
    });
    __syncthreads();
    float2 a[P], b[P];
    own<V>(m0, t, a);
    own<V>(m1, t, b);
    const T *const src[2] = {(const T *)p.x, (const T *)p.dy};
    T *dx = (T *)p.dx;
    const uint32_t limit = drop_limit(p.rng.threshold);
    constexpr bool on = DROP != 0;
    if (t.ty >= 0)
        stream<T, PLAIN, 2, DROP || !PLAIN ? kFewerUnroll : kBackwardUnroll>(g, t, src, p.vec, Nothing(), [&](int64_t e, float2 (&v)[2][P], uint32_t bits) {
        uint32_t r[P];
        if (on) draw(philox, (uint64_t)e, r);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float2 da = grad_a<ACT>(v[0][j], v[1][j], f.nmean[j], f.mul[j], f.add[j], on, on ? r[j] : 0,
                                               limit, p.rng.scale);
            v[0][j] = fma2(v[0][j], b[j], fma2(da, f.mul[j], a[j]));
        }
        if (PLAIN) store_vec(dx + e, true, v[0]);
        else if (bits == ~0u) store_vec(dx + e, p.vec, v[0]);
        else store_some(dx + e, bits, v[0]);
    });
    __syncthreads();
}

template <typename T, bool PLAIN, int ACT, int DROP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    gn_back_fused_kernel(const __grid_constant__ GnGeom g, const __grid_constant__ Params p) {
    const BwdShared sh(g);
    griddep_launch_dependents();
    Shares<PLAIN> shares(g, p);
    Share t;
    int turn = 0;
    cluster_arrive();   // every block of the cluster runs before any stores to it: its push waits
    const int rank = cluster_ctarank();
    const Philox<DROP == 1> philox(p.rng);
    const float inv = (float)(1.0 / ((double)g.S * g.Cg));
    for (int64_t s = blockIdx.y; s < p.strips; s += gridDim.y) {
        shares.get(s, t);
        float4 *pushed = sh.pushed + turn * g.cluster * sh.groups;
        turn ^= 1;
        const Coef<kVec<T>> f(g, p, shares, t, sh);
        block_sums<T, PLAIN, ACT, DROP>(
            g, p, t, f, sh, philox,
            [&] {
                if (s == blockIdx.y) cluster_wait();
            },
            [&](int lg, int lane, int lanes, float2 v) {
                for (int i = lane; i < g.cluster; i += lanes)
                    push(pushed + rank * sh.groups + lg, i, make_float4(v.x, v.y, 0.f, 0.f));
            });
        cluster_arrive();
        cluster_wait();
        for (int lg = threadIdx.x; lg < t.groups; lg += kThreads)
            sh.stat[lg] = mul2(join_pushed(sh, pushed, g.cluster, lg), both(inv));
        if (p.dx) grad_rows<T, PLAIN, ACT, DROP>(g, p, shares, t, f, sh, philox);
        else __syncthreads();
    }
}

template <typename T, bool PLAIN, int ACT, int DROP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    gn_back_sums_kernel(const __grid_constant__ GnGeom g, const __grid_constant__ Params p) {
    const BwdShared sh(g);
    griddep_launch_dependents();
    Shares<PLAIN> shares(g, p);
    Share t;
    const Philox<DROP == 1> philox(p.rng);
    for (int64_t s = blockIdx.y; s < p.strips; s += gridDim.y) {
        shares.get(s, t);
        float2 *out = p.sums + (slots_of<PLAIN>(g, t) + blockIdx.x) * g.G;
        const Coef<kVec<T>> f(g, p, shares, t, sh);
        block_sums<T, PLAIN, ACT, DROP>(
            g, p, t, f, sh, philox, [] {},
            [&](int lg, int lane, int, float2 v) {
                if (lane == 0) out[slot_at<PLAIN>(g, t, wrap_group(g, t.first_group + lg))] = v;
            });
        __syncthreads();
    }
}

// f(group of the tile, sums) with an image's parts joined.
template <bool PLAIN, typename F>
__device__ __forceinline__ void join_parts(const GnGeom &g, const Share &t, const BwdShared &sh, const float2 *sums,
                                           F f) {
    const float2 *in = sums + slots_of<PLAIN>(g, t) * g.G;
    float2 *acc = (float2 *)sh.sums;
    const int log = log_lanes_for(g.tile_groups);
    for (int gb = 0; gb < t.groups; gb += kThreads >> log) {
        const int here = t.groups - gb < kThreads >> log ? t.groups - gb : kThreads >> log;
        const int slices = 1 << log, slice = threadIdx.x / here, lg = gb + threadIdx.x - slice * here;
        float2 s = both(0.f);
        if (slice < slices) {
            const int gi = wrap_group(g, t.first_group + lg), parts = parts_of<PLAIN>(g, t, gi);
            const float2 *q = in + gi;
#pragma unroll 8
            for (int i = slice; i < parts; i += slices) s = add2(s, q[(int64_t)i * g.G]);
            acc[threadIdx.x] = s;
        }
        __syncthreads();
        if (threadIdx.x < here) {
            for (int i = 1; i < slices; ++i) s = add2(s, acc[i * here + threadIdx.x]);
            f(lg, s);
        }
        __syncthreads();
    }
}

template <typename T, bool PLAIN, int ACT, int DROP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    gn_back_apply_kernel(const __grid_constant__ GnGeom g, const __grid_constant__ Params p) {
    const BwdShared sh(g);
    griddep_launch_dependents();
    Shares<PLAIN> shares(g, p);
    Share t;
    const Philox<DROP == 1> philox(p.rng);
    const float inv = (float)(1.0 / ((double)g.S * g.Cg));
    bool waited = false;
    for (int64_t s = blockIdx.y; s < p.strips; s += gridDim.y) {
        shares.get(s, t);
        const Coef<kVec<T>> f(g, p, shares, t, sh);
        if (!waited) griddep_wait();
        waited = true;
        join_parts<PLAIN>(g, t, sh, p.sums, [&](int lg, float2 v) { sh.stat[lg] = mul2(v, both(inv)); });
        grad_rows<T, PLAIN, ACT, DROP>(g, p, shares, t, f, sh, philox);
    }
    if (!waited) griddep_wait();
}

// dw and db: the images', chunks' and copies' parts joined, 16 channels to a
// block, its threads 64 rows of them.
constexpr int kParamThreads = 1024, kParamChannels = 16;
__global__ void __launch_bounds__(kParamThreads)
    gn_back_params_kernel(const __grid_constant__ GnGeom g, const __grid_constant__ Params p) {
    __shared__ float2 sums[kParamThreads];
    griddep_wait();
    const int in = threadIdx.x % kParamChannels, row = threadIdx.x / kParamChannels;
    const int64_t rows = g.N * g.chunks * g.copies;
    for (int64_t c0 = (int64_t)blockIdx.x * kParamChannels; c0 < g.C; c0 += (int64_t)gridDim.x * kParamChannels) {
        const int64_t c = c0 + in;
        float2 s = both(0.f);
        if (c < g.C && g.copies == 1) {
#pragma unroll 8
            for (int64_t r = row; r < rows; r += kParamThreads / kParamChannels) s = add2(s, p.chan[r * g.C + c]);
        } else if (c < g.C) {   // by position: an image's head moves its channels
            for (int64_t r = row; r < rows; r += kParamThreads / kParamChannels) {
                const int64_t at = c + ((r / ((int64_t)g.chunks * g.copies) * g.E) & (g.V - 1));
                s = add2(s, p.chan[r * g.C + (at < g.C ? at : at - g.C)]);
            }
        }
        sums[threadIdx.x] = s;
        __syncthreads();
        if (threadIdx.x < 32 * kParamChannels) {   // one warp per channel, two rows to a lane
            const int ch = threadIdx.x / 32, lane = threadIdx.x % 32;
            s = add2(sums[lane * kParamChannels + ch], sums[(lane + 32) * kParamChannels + ch]);
            s.x = group_sum(s.x, 32);
            s.y = group_sum(s.y, 32);
            if (lane == 0 && c0 + ch < g.C) {
                if (p.dbias) put_param(p.dbias, c0 + ch, p.param_dtype, s.x);
                if (p.dweight) put_param(p.dweight, c0 + ch, p.param_dtype, s.y);
            }
        }
        __syncthreads();
    }
}

// ---- host -------------------------------------------------------------------

template <int V>
struct Int {
    static constexpr int value = V;
};

// f(activation, dropout, plain) with each as a type; dropout: 0 none, 1 with a
// seed given, 2 with one that may lie on the device.  (1 makes the training
// case's two calls 54 us in place of 57; tensors that are not plain do with 2.)
template <typename F>
ct_status by_act(const GnArgs &a, bool plain, F f) {
    auto by_drop = [&](auto act) {
        if (!plain) return a.drop ? f(act, Int<2>(), Int<0>()) : f(act, Int<0>(), Int<0>());
        if (!a.drop) return f(act, Int<0>(), Int<1>());
        return a.rng.dev ? f(act, Int<2>(), Int<1>()) : f(act, Int<1>(), Int<1>());
    };
    if (a.act == CT_ACT_RELU) return by_drop(Int<CT_ACT_RELU>());
    if (a.act == CT_ACT_SILU) return by_drop(Int<CT_ACT_SILU>());
    if (a.act == CT_ACT_GELU) return by_drop(Int<CT_ACT_GELU>());
    return by_drop(Int<CT_ACT_IDENTITY>());
}

Params params_of(const GnGeom &g, const GnArgs &a) {
    Params p = {};
    p.x = a.x; p.dy = a.dy; p.weight = a.weight; p.bias = a.bias;
    p.y = a.y; p.dx = a.dx; p.dweight = a.dweight; p.dbias = a.dbias;
    p.mean = a.mean; p.rstd = a.rstd;
    p.eps = a.eps;
    p.param_dtype = a.param_dtype;
    p.rng = a.rng;
    p.strips = g.N * g.ctiles;
    p.vec = (((uintptr_t)a.x | (uintptr_t)a.dy | (uintptr_t)a.y | (uintptr_t)a.dx) & 15) == 0;
    return p;
}

// Launch with clusters along x; `follows`: it may start while the launch
// before it, of the same call, still runs.
template <typename K>
ct_status launch(K kernel, const GnGeom &g, const Params &p, dim3 grid, int threads, int cluster, size_t smem,
                 bool follows, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (follows) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kernel, g, p) != cudaSuccess) {
        cudaGetLastError();
        return CT_ERR_DEVICE;
    }
    return CT_OK;
}

dim3 grid_of(const GnGeom &g) {
    const int64_t strips = g.N * g.ctiles;
    return dim3((unsigned)g.chunks, (unsigned)(strips < 65535 ? strips : 65535));
}

template <typename T>
ct_status forward_t(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    Params p = params_of(g, a);
    p.part = (float4 *)a.ws;
    const dim3 grid = grid_of(g);
    const size_t smem = forward_smem(g);
    return by_act(a, p.vec && g.wraps == 1 && g.ctiles == 1, [&](auto act, auto drop, auto plain) {
        constexpr int kAct = decltype(act)::value, kDrop = decltype(drop)::value;
        constexpr bool kPlain = decltype(plain)::value != 0;
        static std::atomic<int> ready[3][64];
        if (g.cluster > 0) {
            auto fused = gn_fused_kernel<T, kPlain, kAct, kDrop>;
            if (!allow_smem(fused, ready[0], kMaxSmem)) return CT_ERR_DEVICE;
            return launch(fused, g, p, grid, kThreads, g.cluster, smem, false, st);
        }
        auto stats = gn_stats_kernel<T, kPlain>;
        auto apply = gn_apply_kernel<T, kPlain, kAct, kDrop>;
        if (!allow_smem(stats, ready[1], kMaxSmem) || !allow_smem(apply, ready[2], kMaxSmem)) return CT_ERR_DEVICE;
        const ct_status s = launch(stats, g, p, grid, kThreads, 1, smem, false, st);
        return s == CT_OK ? launch(apply, g, p, grid, kThreads, 1, smem, true, st) : s;
    });
}

template <typename T>
ct_status backward_t(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    Params p = params_of(g, a);
    const bool params = a.dweight || a.dbias;
    p.sums = (float2 *)a.ws;
    if (params) p.chan = p.sums + gn_sums(g);
    const dim3 grid = grid_of(g);
    const size_t smem = backward_smem(g);
    return by_act(a, p.vec && g.wraps == 1 && g.ctiles == 1, [&](auto act, auto drop, auto plain) {
        constexpr int kAct = decltype(act)::value, kDrop = decltype(drop)::value;
        constexpr bool kPlain = decltype(plain)::value != 0;
        static std::atomic<int> ready[3][64];
        ct_status s = CT_OK;
        if (g.N == 0) {
            // nothing to sum: the parameters' gradients are 0
        } else if (g.cluster > 0) {
            auto fused = gn_back_fused_kernel<T, kPlain, kAct, kDrop>;
            if (!allow_smem(fused, ready[0], kMaxSmem)) return CT_ERR_DEVICE;
            s = launch(fused, g, p, grid, kThreads, g.cluster, smem, false, st);
        } else {
            auto sums = gn_back_sums_kernel<T, kPlain, kAct, kDrop>;
            auto apply = gn_back_apply_kernel<T, kPlain, kAct, kDrop>;
            if (!allow_smem(sums, ready[1], kMaxSmem) || !allow_smem(apply, ready[2], kMaxSmem)) return CT_ERR_DEVICE;
            s = launch(sums, g, p, grid, kThreads, 1, smem, false, st);
            if (s == CT_OK && a.dx) s = launch(apply, g, p, grid, kThreads, 1, smem, true, st);
        }
        if (s == CT_OK && params) {
            const int64_t blocks = ceil_div(g.C, kParamChannels);
            s = launch(gn_back_params_kernel, g, p, dim3(blocks < 2048 ? (unsigned)blocks : 2048u), kParamThreads, 1, 0,
                       g.N > 0, st);
        }
        return s;
    });
}

}  // namespace
}  // namespace ct
