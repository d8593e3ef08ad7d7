// Rotary positions: arguments, shared by the C entry point and the kernels.
#pragma once

#include <stdint.h>

#include "ct_divmagic.h"
#include "ct_internal.h"

namespace ct {

constexpr int kRotaryMaxPairs = 256;

struct RotaryParams {
    const void *x, *positions;
    void *y;
    int64_t N, S, H, D;
    int64_t xs[3], ys[3];        // strides of image, pixel and head, in elements
    int64_t grid[3];             // pixels along each axis; positions that are not given are the indices
    int64_t pos_image;           // elements from an image's positions to the next one's
    int32_t axes, rot;           // rot: elements of a head that are rotated
    int32_t first[3];            // each axis' first pair
    int32_t pos_type;            // ct_position_type
    float sign;                  // -1: the inverse
    float near;                  // positions up to it take frequencies of two floats; -1: none does
    int32_t small_grid;          // all indices of the grid are
    // set by rotary_run
    int32_t items;               // of a head, each one thread's
    int32_t groups, per;         // heads are cut into groups of `per`, one thread each
    int64_t threads;             // in all
    int32_t small;               // every index below fits 31 bits: divisions by multiplication
    DivMagic by_items, by_groups, by_s, by_grid[3];
    // Frequency of each pair / 2 pi, also as two floats (high, low).
    double turns[kRotaryMaxPairs];
    alignas(16) float parts[kRotaryMaxPairs][2];
};

ct_status rotary_run(int dtype, int pairs, RotaryParams &p, cudaStream_t st);

}  // namespace ct
