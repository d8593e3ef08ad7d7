// Geometry of a channels-last group norm, shared by the C entry points and
// the kernels.
//
// The elements of image n are one contiguous run of S*C; kernels read it as
// aligned vectors of eight elements counted from the run's start rounded down
// to a multiple of eight (`head` elements before it belong to the previous
// image).  A "row" is the shortest run of whole pixels that is a multiple of
// eight elements: L = C * 8 / gcd(C, 8), so a thread that keeps its column
// and walks the rows always meets the same eight channels, for any C, and
// holds its channels' coefficients and sums in registers.
#pragma once

#include <stdint.h>

#include "ct_internal.h"
#include "philox.cuh"

namespace ct {

struct GnGeom {
    int64_t N, S, E;       // images, pixels per image, elements per image (S*C)
    int32_t C, G, Cg;
    int32_t wraps;         // pixels per row, L / C
    int32_t LV;            // vectors per row, L / 8
    int64_t rows;          // rows that cover any image, head included
    int32_t bx, by;        // a block's threads: columns x rows
    int32_t ctiles;        // column tiles per row
    int64_t rpc;           // rows per chunk
    int32_t chunks;        // chunks per image
    int64_t items;         // N * chunks * ctiles
};

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

GnGeom gn_geom(int64_t N, int64_t S, int64_t C, int64_t G);
size_t gn_forward_ws(const GnGeom &g);
size_t gn_backward_ws(const GnGeom &g);
ct_status gn_forward(const GnGeom &g, const GnArgs &a, cudaStream_t st);
ct_status gn_backward(const GnGeom &g, const GnArgs &a, cudaStream_t st);

ct_status dropout_run(int dtype, const void *x, const void *residual, void *y, int64_t n, const RngArgs &rng,
                      cudaStream_t st);

}  // namespace ct
