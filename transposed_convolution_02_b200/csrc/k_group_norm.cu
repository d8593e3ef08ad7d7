// The group norm's geometry: how images are cut into strips and chunks; and
// what is left of a call on images of no pixels.
#include "ct_cuda_util.h"
#include "group_norm.h"

namespace ct {

namespace {

// The statistics of images without pixels.
__global__ void __launch_bounds__(kThreads) gn_empty_kernel(float *mean, float *rstd, int64_t n, float eps) {
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        if (mean) mean[i] = 0.f;
        if (rstd) rstd[i] = 1.f / sqrtf(eps);
    }
}

}  // namespace

GnGeom gn_geom(int64_t N, int64_t S, int64_t C, int64_t G, int dtype, int tensors) {
    GnGeom g = {};
    const int size = dtype == CT_F32 ? 4 : 2;
    const int64_t slots = 148 * kBlocksPerSm;   // resident blocks
    g.V = 16 / size;
    g.N = N; g.S = S; g.E = S * C;
    g.C = (int32_t)C; g.G = (int32_t)G; g.Cg = (int32_t)(C / G);
    int64_t d = g.V;
    while (C % d != 0) d /= 2;
    g.wraps = (int32_t)(g.V / d);
    g.LV = (int32_t)(C / d);
    g.full_rows = g.E / g.V / g.LV;
    g.full_rest = (int32_t)(g.E / g.V % g.LV);
    // the head of an image whose elements do not start at a multiple of V can
    // take one more row
    const int64_t head = g.E % g.V == 0 || N <= 1 ? 0 : g.V - 1;
    g.rows = ceil_div(head + g.E, (int64_t)g.LV * g.V);
    if (g.rows < 1) g.rows = 1;
    const int64_t image = g.E * size * tensors;
    g.ctiles = (int32_t)ceil_div(g.LV, (int64_t)kMaxColumns);
    g.bx = (int32_t)ceil_div(g.LV, (int64_t)g.ctiles);
    int64_t by = kThreads / g.bx;
    if (by > g.rows) by = g.rows;
    g.by = (int32_t)by;
    g.by_bx = make_magic((uint32_t)g.bx);
    g.by_by = make_magic((uint32_t)g.by);
    g.by_cg = make_magic((uint32_t)g.Cg);
    const int64_t width = (int64_t)g.bx * g.V;   // positions of a tile
    g.by_tile = make_magic((uint32_t)width);
    g.copies = g.slots = 1;
    g.tile_groups = g.G;
    if (g.ctiles > 1) {
        // as many as `width` neighbours meet, the first and the last cut
        const int64_t met = (width + 2 * (int64_t)g.Cg - 2) / g.Cg;
        if (met < g.G) g.tile_groups = (int32_t)met;
        // an image's head moves its channels along the row by less than C, so S
        // pixels take S + 1 copies there; a group that the row's ends cut has a
        // run more than copies, and a run of Cg positions lies in at most
        // ceil((Cg - 1) / width) + 1 tiles
        if (g.wraps > 1) g.copies = (int32_t)(S + 1 < g.wraps ? S + 1 : g.wraps);
        const int64_t runs = g.wraps > 1 && g.Cg > 1 ? g.copies + 1 : g.copies;
        const int64_t tiles = runs * (ceil_div((int64_t)g.Cg - 1, width) + 1);
        g.slots = (int32_t)(tiles < g.ctiles ? tiles : g.ctiles);
    }

    // One launch: a cluster of up to 8 blocks per strip, where that fills half
    // of the GPU or the tensor is small, and no group spans column tiles.
    // (Clusters of 16 are placed so slowly that [16,32x32,512] bf16 took 33 us
    // in place of 22.)
    const int64_t strips = N * g.ctiles;
    const bool whole = g.ctiles == 1 || (g.wraps == 1 && g.bx * g.V % g.Cg == 0);
    int64_t cluster = 1;
    while (cluster < 8 && cluster * 2 * strips <= slots && cluster * 2 * by <= g.rows &&
           cluster * 2 * groups_max(g) <= kMaxPushed)
        cluster *= 2;
    if (whole && g.rows < (int64_t(1) << 30) && (N * image <= kSmallBytes || 2 * cluster * strips >= slots) &&
        image <= cluster * kClusterBytes) {
        g.cluster = (int32_t)cluster;
        g.chunks = g.cluster;
        g.rpc = (int32_t)ceil_div(g.rows, cluster);
        return g;
    }
    // Two launches, of one round of resident blocks; more where a thread would
    // sum too many rows one after the other, fewer where it had less than two.
    int64_t chunks = strips < slots ? slots / (strips < 1 ? 1 : strips) : 1;
    const int64_t useful = ceil_div(g.rows, by * 2), least = ceil_div(g.rows, by * kMaxRows);
    if (chunks > useful) chunks = useful;
    if (chunks < least) chunks = least;
    if (chunks > int64_t(1) << 30) chunks = int64_t(1) << 30;
    g.rpc = (int32_t)ceil_div(g.rows, chunks);
    g.chunks = (int32_t)ceil_div(g.rows, (int64_t)g.rpc);
    return g;
}

// No product here leaves 64 bits: slots * G <= 19 C (a tile has more than 512
// positions where there are several), N C <= 2^54, N S C <= 2^60, and chunks is
// at most 592 / (N ctiles) or S / 1024 + 1.
int64_t gn_sums(const GnGeom &g) { return g.cluster > 0 ? 0 : g.N * g.slots * g.chunks * g.G; }

size_t gn_forward_ws(const GnGeom &g) { return g.E == 0 ? 0 : (size_t)gn_sums(g) * 16; }

size_t gn_backward_ws(const GnGeom &g) {
    return g.E == 0 ? 0 : (size_t)(gn_sums(g) + g.N * g.chunks * g.copies * g.C) * 8;
}

// Images without pixels: no kernel walks them (their number is bounded by no
// memory), and no statistics are read.
ct_status gn_forward(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    if (g.E == 0) {
        const int64_t n = g.N * g.G, blocks = ceil_div(n, (int64_t)kThreads);
        if (n == 0 || (!a.mean && !a.rstd)) return CT_OK;
        gn_empty_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), kThreads, 0, st>>>(a.mean, a.rstd, n, a.eps);
        return launch_status();
    }
    if (a.dtype == CT_F32) return gn_forward_f32(g, a, st);
    if (a.dtype == CT_F16) return gn_forward_f16(g, a, st);
    return gn_forward_bf16(g, a, st);
}

ct_status gn_backward(const GnGeom &geom, const GnArgs &a, cudaStream_t st) {
    GnGeom g = geom;
    if (g.E == 0) g.N = 0;
    if (a.dtype == CT_F32) return gn_backward_f32(g, a, st);
    if (a.dtype == CT_F16) return gn_backward_f16(g, a, st);
    return gn_backward_bf16(g, a, st);
}

}  // namespace ct
