// AdamW over many tensors at once, and their gradients' norm: arguments shared
// by the C entry points and the kernels.
//
// All tensors are cut into blocks of 256 elements, one warp's work; a launch
// has a table of its tensors among its arguments, so that a step copies
// nothing to the device and a captured one carries its addresses along.
#pragma once

#include <stdint.h>

#include "ct_internal.h"
#include "philox.cuh"

namespace ct {

constexpr int kBlock = 256;           // elements under one scale of 8-bit states
constexpr int kFewTensors = 32;       // of a launch's table, three sizes: 1.8, 7 and 28 KB of arguments
constexpr int kSomeTensors = 128;
constexpr int kManyTensors = 512;
constexpr int kNormBlocks = 148 * 4;  // of a launch of the norm: partial sums, whatever the device

struct TensorEntry {
    void *param;
    const void *grad;
    int64_t n;
    int64_t first;     // block of the launch that it starts at
    int64_t state;     // block of the states
    int64_t master;    // block of the masters
    float decay;
    uint32_t kind;     // param's ct_dtype, grad's << 2, and whether they lie on whole vectors: 16, 32
};
enum : uint32_t { kParamVec = 16, kGradVec = 32 };

template <int N>
struct TensorTable {
    TensorEntry t[N];
    int32_t count;
    int64_t blocks;
};

struct AdamWParams {
    float beta1, beta2, rest1, rest2, eps;     // rest: 1 - beta
    float lr, lr_c1, root_c2;                  // lr / (1 - beta1^t), (1 - beta2^t)^-1/2
    float log1, log2;                          // natural logarithms of the betas, for a step that lies on the device
    uint64_t step;
    const float *lr_dev, *grad_scale;
    const int64_t *step_dev;
    void *m, *v;
    float *m_scale, *v_scale, *master;
    RngArgs rng;
};

// The host fills a table and launches it whenever it is full.
ct_status adamw_run(const ct_adamw_desc *d, int64_t count, const ct_param *shapes, void *const *params,
                    const void *const *grads, AdamWParams &p, cudaStream_t st);
ct_status grad_norm_run(int64_t count, const ct_param *shapes, const void *const *grads, double max_norm, float *norm,
                        float *scale, double *ws, cudaStream_t st);

inline int64_t norm_partials(int64_t count) { return (ceil_div(count, (int64_t)kManyTensors) + 1) * kNormBlocks; }

}  // namespace ct
