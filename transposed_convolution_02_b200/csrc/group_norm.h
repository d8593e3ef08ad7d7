// Geometry of a channels-last group norm, shared by the C entry points and
// the kernels.
//
// The elements of image n are one contiguous run of S*C; kernels read it as
// aligned vectors of 16 bytes (V elements: 8 of a 16-bit type, 4 of fp32)
// counted from the run's start rounded down to a multiple of V (`head`
// elements before it belong to the previous image).  A "row" is the shortest
// run of whole pixels that is a multiple of V elements, L = C * V / gcd(C, V):
// a thread that keeps its column and walks the rows always meets the same V
// channels, for any C, and holds its channels' coefficients and sums in
// registers.  Rows wider than a block's threads are cut into column tiles; a
// tile of an image is a "strip", and every strip is cut into `chunks` runs of
// `rpc` rows, one to a block.  Divisions by these sizes are multiplications by
// host-made factors: a block's fixed work counts where images are small.
#pragma once

#include <stdint.h>

#include "ct_divmagic.h"
#include "ct_internal.h"
#include "philox.cuh"

namespace ct {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 2;
// Vectors in flight per thread and tensor.  Backward, plain kernels without a
// mask take 6 (186 us in place of 198 at [16,112x112,512] fp16), the others 4
// (with a mask 6 spill: 39 us in place of 34 at [16,32x32,512] bf16; general
// kernels grow: 14.5 us in place of 11.8 at [2,13x17,65] fp32).
constexpr int kForwardUnroll = 8, kBackwardUnroll = 6, kFewerUnroll = 4;
constexpr int kMaxColumns = 256;           // vectors across a column tile
constexpr int kMaxPushed = 1024;           // group sums that a block takes from its cluster
constexpr int kMaxSmem = 144 * 1024;       // of any geometry: 2048 positions, 2049 groups
constexpr int64_t kSmallBytes = 4 << 20;   // of the tensors read, that a cluster per strip may always take
constexpr int64_t kClusterBytes = 1 << 20; // of an image per block of its cluster
constexpr int64_t kMaxRows = 1024;         // vectors that a thread sums one after the other

struct GnGeom {
    int64_t N, S, E;       // images, pixels per image, elements per image (S*C)
    int32_t C, G, Cg, V;
    int32_t wraps;         // pixels per row, L / C
    int32_t LV;            // vectors per row, L / V
    int64_t full_rows;     // rows of E / V vectors that are whole
    int32_t full_rest;     // and the vectors beyond them
    int64_t rows;          // rows that cover any image, head included
    int32_t bx, by;        // a block's threads: columns x rows
    int32_t ctiles;        // column tiles per row
    int32_t rpc, chunks;   // rows per chunk; chunks per strip
    int32_t cluster;       // one launch, a cluster of that many blocks per strip; 0: two launches
    // With several column tiles (all 1 with one): copies of the channels along a
    // row that an image can have values in, and the most tiles that a group's
    // channels lie in there. The workspace holds a slot per group and tile of
    // it, and per channel and copy.
    int32_t copies, slots;
    int32_t tile_groups;   // groups that a tile meets at most; all with one tile
    DivMagic by_bx, by_by, by_cg, by_tile;   // divisors bx, by, Cg, bx * V
};

// Groups that a column tile can meet.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int groups_max(const GnGeom &g) {
    return g.G < g.bx * g.V + 1 ? g.G : g.bx * g.V + 1;
}

struct GnArgs {
    int dtype, param_dtype, act;
    float eps;
    const void *x, *dy, *weight, *bias;
    void *y, *dx, *dweight, *dbias;
    float *mean, *rstd;    // [N, G]
    bool drop;
    RngArgs rng;
    float *ws;
};

// `tensors`: how many tensors of x's size a pass reads: 1 forward, 2 backward.
GnGeom gn_geom(int64_t N, int64_t S, int64_t C, int64_t G, int dtype, int tensors);
int64_t gn_sums(const GnGeom &g);   // group sums in the workspace, before a backward's channel sums
size_t gn_forward_ws(const GnGeom &g);
size_t gn_backward_ws(const GnGeom &g);
ct_status gn_forward(const GnGeom &g, const GnArgs &a, cudaStream_t st);
ct_status gn_backward(const GnGeom &g, const GnArgs &a, cudaStream_t st);
ct_status gn_forward_f32(const GnGeom &g, const GnArgs &a, cudaStream_t st);
ct_status gn_forward_f16(const GnGeom &g, const GnArgs &a, cudaStream_t st);
ct_status gn_forward_bf16(const GnGeom &g, const GnArgs &a, cudaStream_t st);
ct_status gn_backward_f32(const GnGeom &g, const GnArgs &a, cudaStream_t st);
ct_status gn_backward_f16(const GnGeom &g, const GnArgs &a, cudaStream_t st);
ct_status gn_backward_bf16(const GnGeom &g, const GnArgs &a, cudaStream_t st);

ct_status dropout_run(int dtype, const void *x, const void *residual, void *y, int64_t n, const RngArgs &rng,
                      cudaStream_t st);

}  // namespace ct
