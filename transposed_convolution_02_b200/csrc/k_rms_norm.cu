// The root-mean-square norm's geometry: how many threads share a row, and what
// each of them holds.
#include "rms_norm.h"

namespace ct {

namespace {

int64_t pow2_at_least(int64_t n) {
    int64_t p = 1;
    while (p < n) p *= 2;
    return p;
}

// The least of `of` (ascending, 0 at its end) that makes `tpr` threads hold n; 0: none.
int least_k(const int *of, int tpr, int64_t n) {
    for (; *of; ++of)
        if ((int64_t)tpr * *of >= n) return *of;
    return 0;
}

constexpr int kMaxTpr = 512;

// `want`: vectors per thread where a row leaves the choice; `least`: threads
// that a row has at least, if it has as many vectors; `most`: threads of a block
// that have no more vectors than that.
void spread(RmsGeom &g, int64_t n, int want, int least, const int *of, int most) {
    int64_t tpr = pow2_at_least((n + want - 1) / want);
    const int64_t all = n < least ? pow2_at_least(n) : least;
    if (tpr < all) tpr = all;
    if (tpr > most) tpr = kMaxTpr;
    g.tpr = (int)tpr;
    g.K = least_k(of, g.tpr, n);
    if (g.K == 0) g.tpr = kMaxTpr;
    g.threads = g.tpr > 256 ? g.tpr : 256;
}

}  // namespace

RmsGeom rms_forward_geom(const RmsArgs &a, bool aligned) {
    static const int vec16[] = {1, 2, 4, 8, 0}, ones[] = {1, 2, 4, 8, 32, 0}, ones128[] = {4, 8, 32, 0};
    RmsGeom g = {};
    const int V = a.dtype == CT_F32 ? 4 : 8;
    g.vec = aligned && a.C % V == 0;
    const bool blocks = a.scale && a.block != 0 && a.block < a.C;
    if (g.vec) {
        // 16 elements a thread (32: [32768,4096] fp16 with a residual 196 us in
        // place of 160; 8: e4m3 349 in place of 194); eight neighbours at least
        // read 128 bytes together; a block's channels lie in one warp
        const int lanes = blocks && a.block / V > 8 ? a.block / V : 8;
        spread(g, a.C / V, kRmsFewElements / V, lanes, vec16, 512);
    } else {
        spread(g, a.C, 8, 32, blocks && a.block == 128 ? ones128 : ones, 1024);
    }
    g.blocks = ceil_div(a.rows, (int64_t)(g.threads / g.tpr));
    if (g.blocks > 0x7FFFFFFF) g.blocks = 0x7FFFFFFF;
    // With one tensor to read and one to write, blocks that stay keep more bytes
    // in flight ([32768,4096] bf16 96 us, 118 without; with a residual 176 to
    // 190, 157 without; e4m3 with a residual 243, 149 without).  1024 threads an
    // SM, as the registers let them be.
    const int64_t staying = 148 * 1024 / g.threads;
    if (g.vec && g.K > 0 && g.K * V <= kRmsFewElements && !a.residual && !a.scale && g.blocks >= 2 * staying)
        g.ring = staying;
    return g;
}

// dweight's partial sums.  Rows in registers: one of each block, all resident
// at once.  Rows that are walked: enough for a round of blocks of 256 columns.
int64_t rms_parts(int64_t rows, int64_t C) {
    const int64_t most = C <= 16384 ? 148 * 4 : 148 * 8 * 256 / C;
    const int64_t n = C <= 16384 ? rows : ceil_div(rows, (int64_t)32);
    const int64_t parts = n < most ? n : most;
    return parts < 1 ? 1 : parts;
}

RmsGeom rms_backward_geom(const RmsArgs &a, bool aligned) {
    static const int vec8[] = {1, 2, 4, 0}, vec4[] = {1, 2, 4, 8, 0}, ones[] = {1, 2, 4, 8, 32, 0};
    RmsGeom g = {};
    const int V = a.dtype == CT_F32 ? 4 : 8;
    g.vec = aligned && a.C % V == 0;
    if (g.vec) spread(g, a.C / V, 2, 8, V == 8 ? vec8 : vec4, 512);
    else spread(g, a.C, 8, 32, ones, 512);
    const int64_t rounds = ceil_div(a.rows, (int64_t)(g.threads / g.tpr));
    // one round of resident blocks, as the ring lets them be
    int64_t parts = rms_parts(a.rows, a.C);
    if (g.vec && g.K > 0) {
        const int64_t ring = (int64_t)rms_stages(g.K) * (a.dsum ? 3 : 2) * g.K * g.threads * 16 + 2048;
        int64_t resident = (228 * 1024) / ring;
        if (resident > 2) resident = 2;
        if (parts > 148 * resident) parts = 148 * resident;
    }
    g.blocks = rounds < parts ? rounds : parts;
    if (g.blocks < 1) g.blocks = 1;
    return g;
}

namespace {

bool all_aligned(const RmsArgs &a) {
    const uintptr_t p = (uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.weight | (uintptr_t)a.sum |
                        (uintptr_t)a.dy | (uintptr_t)a.dsum | (uintptr_t)a.dx;
    // codes: a vector's worth of them is half as long as a vector, or a quarter
    return (p & 15) == 0 && ((uintptr_t)a.y & (a.scale ? 7 : 15)) == 0;
}

}  // namespace

ct_status rms_forward(const RmsArgs &a, cudaStream_t st) {
    const RmsGeom g = rms_forward_geom(a, all_aligned(a));
    if (a.dtype == CT_F32) return rms_forward_f32(a, g, st);
    if (a.dtype == CT_F16) return rms_forward_f16(a, g, st);
    return rms_forward_bf16(a, g, st);
}

ct_status rms_backward(const RmsArgs &a, cudaStream_t st) {
    const RmsGeom g = rms_backward_geom(a, all_aligned(a));
    if (a.dtype == CT_F32) return rms_backward_f32(a, g, st);
    if (a.dtype == CT_F16) return rms_backward_f16(a, g, st);
    return rms_backward_bf16(a, g, st);
}

}  // namespace ct
