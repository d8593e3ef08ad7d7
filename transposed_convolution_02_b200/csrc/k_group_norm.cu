// The group norm's geometry: how images are cut into waves, strips and chunks.
#include "group_norm.h"

namespace ct {

GnGeom gn_geom(int64_t N, int64_t S, int64_t C, int64_t G, int dtype, int tensors) {
    GnGeom g = {};
    const int size = dtype == CT_F32 ? 4 : 2;
    const int64_t slots = 148 * (tensors == 1 ? kForwardBlocks : kBackwardBlocks);
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

    // Fused: as many blocks to a cluster as fill the GPU, up to 16, each thread
    // with a row or more.  Not where a group spans column tiles, where the
    // images under work at a time would not stay in L2, or where the clusters
    // would leave much of the GPU idle with long work to do.
    const int64_t strips = N * g.ctiles;
    int64_t cluster = 1;
    while (cluster < CT_GN_FCL && cluster * 2 * strips <= slots && cluster * 2 * by <= g.rows &&
           cluster * 2 * groups_max(g) <= kMaxPushed)
        cluster *= 2;
    const int64_t at_once = strips < slots / cluster ? strips : slots / cluster;
    const bool whole = g.ctiles == 1 || (g.wraps == 1 && g.bx * g.V % g.Cg == 0);
    if (whole && at_once * image / g.ctiles <= kWaveBytes && g.rows < (int64_t(1) << 30) &&
        (2 * cluster * strips >= slots || image * N <= (4 << 20))) {
        g.fused = true;
        g.wave = N;
        g.cluster = (int32_t)cluster;
        g.rpc = (int32_t)ceil_div(g.rows, cluster);
        g.chunks = g.cluster;
        g.parts = 1;
        return g;
    }
    // Two launches: waves of equal size, and one round of resident blocks over
    // a wave.
    int64_t wave = image > 0 ? kWaveBytes / image : N;
    if (wave < 1) wave = 1;
    g.wave = N > 0 ? ceil_div(N, ceil_div(N, wave)) : 1;
    int64_t chunks = g.wave * g.ctiles < slots ? slots / (g.wave * g.ctiles) : 1;
    const int64_t useful = ceil_div(g.rows, by * 2), least = ceil_div(g.rows, int64_t(1) << 30);
    if (chunks > useful) chunks = useful;
    if (chunks < least) chunks = least;
    g.cluster = 1;
    while (g.cluster < CT_GN_CL && g.cluster * 2 <= chunks && g.cluster * 2 * groups_max(g) <= kMaxPushed) g.cluster *= 2;
    g.chunks = (int32_t)(chunks / g.cluster * g.cluster);
    g.rpc = (int32_t)ceil_div(g.rows, (int64_t)g.chunks);
    g.parts = g.chunks / g.cluster;
    int64_t finer = chunks * CT_GN_APPLY;
    if (finer > useful) finer = useful;
    if (finer < chunks) finer = chunks;
    g.apply_rpc = (int32_t)ceil_div(g.rows, finer);
    g.apply_chunks = (int32_t)ceil_div(g.rows, (int64_t)g.apply_rpc);
    return g;
}

size_t gn_forward_ws(const GnGeom &g) {
    return g.fused ? 0 : (size_t)(g.N * g.ctiles * g.parts * g.G) * sizeof(float4);
}

size_t gn_backward_ws(const GnGeom &g) {
    return (size_t)(g.N * g.ctiles * ((int64_t)g.parts * g.G + (int64_t)g.chunks * g.C)) * sizeof(float2);
}

ct_status gn_forward(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    if (a.dtype == CT_F32) return gn_forward_f32(g, a, st);
    if (a.dtype == CT_F16) return gn_forward_f16(g, a, st);
    return gn_forward_bf16(g, a, st);
}

ct_status gn_backward(const GnGeom &g, const GnArgs &a, cudaStream_t st) {
    if (a.dtype == CT_F32) return gn_backward_f32(g, a, st);
    if (a.dtype == CT_F16) return gn_backward_f16(g, a, st);
    return gn_backward_bf16(g, a, st);
}

}  // namespace ct
