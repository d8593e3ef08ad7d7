// Root-mean-square norm: arguments and geometry, shared by the C entry points
// and the kernels.
//
// A row (a pixel, a token, a head) of C channels belongs to some lanes of a warp
// or to some warps; a thread holds K vectors of E elements of it in registers, so
// that every tensor is read once.  E is a vector of 16 bytes where the tensors
// start on one, else a single element.  Rows longer than a block holds are walked
// twice by kernels of their own.
#pragma once

#include <stdint.h>

#include "ct_internal.h"

namespace ct {

struct RmsArgs {
    int dtype, param_dtype;      // ct_dtype
    int64_t rows;
    int64_t C;
    float eps;
    int block;                   // channels under one scale; 0: all of a row. (e4m3 only)
    const void *x, *residual, *weight;
    void *y, *sum;               // y: of x's type, or e4m3 codes where `scale` is set
    float *rstd, *scale;
    const void *dy, *dsum;       // backward; x is then what was normed
    const float *rstd_in;
    void *dx, *dweight;
    float *ws;
};

struct RmsGeom {
    bool vec;           // 16-byte vectors, else single elements
    bool shift;         // rows start inside vectors
    int K;              // vectors of a row per thread; 0: the row is walked
    int lanes_log2;     // of a row: 5 where it has whole warps
    int warps;          // of a row
    int rpb;            // rows of a block
    int threads;        // per block
    int64_t blocks;
    int64_t ring;       // blocks of the forward kernel that stays for many rows; 0: not that one
};

// Rows of the backward ring for K vectors a thread.
constexpr int rms_stages(int K) { return K <= 2 ? 4 : K <= 4 ? 2 : 1; }

constexpr int rms_forward_stages(int K) { return K <= 2 ? 4 : 3; }
constexpr int kRmsFewElements = 16;     // of a thread, with which a forward block may have 1024

constexpr int64_t kRmsMaxC = int64_t(1) << 24;

// Where the pointers of a call allow vectors.  The workspace does not depend
// on it: rms_parts is the same for both.
RmsGeom rms_forward_geom(const RmsArgs &a, bool aligned);
RmsGeom rms_backward_geom(const RmsArgs &a, bool aligned);
int64_t rms_parts(int64_t rows, int64_t C);     // partial sums of dweight: rows of C floats in the workspace

ct_status rms_forward(const RmsArgs &a, cudaStream_t st);
ct_status rms_backward(const RmsArgs &a, cudaStream_t st);
ct_status rms_forward_f32(const RmsArgs &a, const RmsGeom &g, cudaStream_t st);
ct_status rms_forward_f16(const RmsArgs &a, const RmsGeom &g, cudaStream_t st);
ct_status rms_forward_bf16(const RmsArgs &a, const RmsGeom &g, cudaStream_t st);
ct_status rms_backward_f32(const RmsArgs &a, const RmsGeom &g, cudaStream_t st);
ct_status rms_backward_f16(const RmsArgs &a, const RmsGeom &g, cudaStream_t st);
ct_status rms_backward_bf16(const RmsArgs &a, const RmsGeom &g, cudaStream_t st);

}  // namespace ct
