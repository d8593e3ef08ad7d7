/*
 * ct.h -- C ABI of the B200 (sm_100a) ONNX ConvTranspose library (libct.so),
 * of the group norm and dropout that follow it in a decoder, and of what stands
 * around the matrix products of a decoder's blocks: root-mean-square norm,
 * rotary positions, and the training step's end (gradient norm, AdamW).
 *
 * The operation (ai.onnx.ConvTranspose README, "Description", "Inputs",
 * "Outputs", "Attributes" and "Type constraints"): Y is the transposed
 * (fractionally strided) convolution of X with W, plus an optional bias B
 * per output channel.  With pad_begin/pad_end resolved per spatial axis a,
 * input position i and kernel tap k land on output position
 *
 *     o_a = i_a * strides_a - pad_begin_a + k_a * dilations_a
 *
 * and Y[n, g*M/group + m, o] is the sum of X[n, g*C/group + c, i] *
 * W[g*C/group + c, m, k] over every (c, i, k) landing on o, plus B[...].
 * The output size per axis is
 *
 *     out_a = strides_a*(in_a - 1) + output_padding_a + (k_a - 1)*dilations_a
 *             + 1 - pad_begin_a - pad_end_a.
 *
 * Two layouts are served:
 *   CT_NCHW  channels-first, as the ai.onnx.ConvTranspose README states it:
 *            X[N, C, D1..Dr], W[C, M/group, k1..kr], Y[N, M, out1..outr].
 *   CT_NHWC  channels-last, as ClikaRT::ops::conv_transpose states it (its
 *            layout paragraph): X[N, D1..Dr, C], W[C, k1..kr, M/group]
 *            (input-channel first), Y[N, out1..outr, M].
 * X, W, B and Y share one element type T in {float32, float16} (README,
 * "Type constraints").  All tensors are dense, row-major, in device memory.
 *
 * Ownership: the caller owns every device buffer and the stream; the library
 * owns only the opaque plan.  No entry point calls a device allocator; the
 * device memory libct.so holds by itself is its code and its file-scope
 * device arrays (the ct_run_noalloc workspace among them), which CUDA loads
 * onto a device with the library's kernels, at the latest on the first call
 * that uses that device.
 * Errors: every entry point returns a ct_status; nothing is thrown across the
 * ABI, nothing is printed.  Validation happens in ct_plan, before any launch.
 * The status classes mirror the error classes of ClikaRT::ops::conv_transpose
 * ("Throws": channel/group arithmetic, span lengths, dtype).
 */
#ifndef CT_H_
#define CT_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define CT_API __attribute__((visibility("default")))
#else
#define CT_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ct_status {
    CT_OK = 0,
    CT_ERR_CHANNELS = 1,   /* C % group != 0, W dims inconsistent with C/group, or bias length != M */
    CT_ERR_SPAN = 2,       /* rank outside 1..3, or an attribute span of the wrong length */
    CT_ERR_DTYPE = 3,      /* element type not float32/float16, or layout unknown */
    CT_ERR_ATTR = 4,       /* stride/dilation/kernel <= 0, output_padding >= max(stride, dilation),
                              kernel_shape != W dims, pads with auto_pad, empty or inconsistent output */
    CT_ERR_ALIGN = 5,      /* a device pointer is not aligned as the chosen kernel requires */
    CT_ERR_NULL = 6,       /* a required pointer is NULL */
    CT_ERR_DEVICE = 7,     /* the current device is not sm_100, or a CUDA launch failed */
    CT_ERR_WORKSPACE = 8,  /* workspace pointer missing although ct_workspace_bytes > 0 */
    CT_ERR_UNSUPPORTED = 9,/* a forced algorithm cannot serve this shape */
    CT_ERR_NOMEM = 10      /* host allocation of the plan failed */
} ct_status;

/* ConvTranspose takes CT_F32 and CT_F16; all other operators also CT_BF16. */
typedef enum ct_dtype { CT_F32 = 0, CT_F16 = 1, CT_BF16 = 2 } ct_dtype;
typedef enum ct_layout { CT_NCHW = 0, CT_NHWC = 1 } ct_layout;

/* auto_pad (README "Attributes"): NOTSET uses pads; SAME_UPPER/SAME_LOWER give
 * out = in * stride with the odd unit of the total padding at the end / the
 * beginning; VALID pads nothing. */
typedef enum ct_autopad {
    CT_AUTOPAD_NOTSET = 0,
    CT_AUTOPAD_SAME_UPPER = 1,
    CT_AUTOPAD_SAME_LOWER = 2,
    CT_AUTOPAD_VALID = 3
} ct_autopad;

/* Kernel selection: CT_ALGO_AUTO lets ct_plan choose; the others force one
 * kernel (for tests) and make ct_plan return CT_ERR_UNSUPPORTED when that
 * kernel cannot serve the shape. */
typedef enum ct_algo {
    CT_ALGO_AUTO = 0,
    CT_ALGO_GENERIC = 1,   /* per-output gather, any shape */
    CT_ALGO_DENSE_TC = 2,  /* fp16 group-1 phase GEMM on tcgen05 tensor cores */
    CT_ALGO_FP32_GEMM = 3, /* fp32 group-1 register-tiled FFMA phase GEMM */
    CT_ALGO_GROUPED = 4,   /* fp16 grouped phase kernel (mma.sync), small per-group slabs */
    CT_ALGO_DENSE_TC_PERTAP = 5, /* fp16 group-1 tcgen05 phase GEMM, one input load per tap
                                    (the general fallback of CT_ALGO_DENSE_TC) */
    CT_ALGO_DENSE_TC_PAIR = 6    /* group-1 phase GEMM, each MMA spanning the two SMs of a CTA
                                    pair (tcgen05 cta_group::2), either layout; fp16 (chosen
                                    automatically for channels-first with one or two spatial
                                    axes) or fp32 as 3xTF32 (TF32 high part and remainder of
                                    both operands, three MMAs per step; chosen automatically
                                    for fp32).  The workspace holds a zero-padded
                                    channels-last copy of X (two planes, high parts and
                                    remainders, for fp32) */
} ct_algo;

/* Activation applied to every output after the bias (ClikaRT::ops::
 * conv_transpose, parameter `activation`, default Identity).  The page does
 * not list the Activation members; this library offers identity and ReLU
 * (max(v, 0)), applied in fp32 before the output is rounded to its dtype.
 * Any other value is CT_ERR_ATTR.  The group norm also takes SILU (v /
 * (1 + exp(-v))) and GELU (v/2 * (1 + erf(v / sqrt 2))). */
typedef enum ct_activation {
    CT_ACT_IDENTITY = 0,
    CT_ACT_RELU = 1,
    CT_ACT_SILU = 2,
    CT_ACT_GELU = 3
} ct_activation;

/* One ConvTranspose call.  Every array has 3 slots; only the first `rank`
 * (and 2*rank for pads) are read. */
typedef struct ct_desc {
    int32_t rank;              /* spatial rank r, 1..3 */
    int32_t dtype;             /* ct_dtype */
    int32_t layout;            /* ct_layout */
    int32_t auto_pad;          /* ct_autopad */
    int64_t N;                 /* batch */
    int64_t C;                 /* input channels */
    int64_t in[3];             /* input spatial sizes D1..Dr */
    int64_t w_dims[5];         /* W's dims as declared: CT_NCHW [C, M/group, k1..kr],
                                  CT_NHWC [C, k1..kr, M/group] */
    int64_t group;
    int64_t bias_len;          /* 0: no bias; else must equal M */
    int64_t strides[3];
    int64_t dilations[3];
    int64_t pads[6];           /* README order: begins of every axis, then ends */
    int64_t output_padding[3];
    int32_t has_kernel_shape;
    int32_t has_output_shape;
    int64_t kernel_shape[3];
    int64_t output_shape[3];
    int32_t algo;              /* ct_algo */
    int32_t activation;        /* ct_activation */
} ct_desc;

typedef struct ct_plan_s ct_plan_t;

/* Resolve the output: Y's dims in the descriptor's layout (rank + 2 entries)
 * and the begin/end pads per axis.  Pure host code, no device touched.
 * Implements the output-size rule above with the auto_pad / output_shape /
 * output_padding rows of the README's "Attributes" table.  Library limits
 * (CT_ERR_ATTR beyond them, so that no size arithmetic overflows int64):
 * N, C, M/group, group, every spatial size, kernel size, stride, dilation,
 * pad and requested output size at most 2^30 in magnitude; X, W and Y each
 * at most 2^60 elements. */
CT_API ct_status ct_output_shape(const ct_desc *desc, int64_t y_dims[5],
                          int64_t pad_begin[3], int64_t pad_end[3]);

/* Validate the descriptor, resolve it, build the stride-phase table and
 * choose a kernel.  Pure host code.  On success *out owns a plan that the
 * caller frees with ct_plan_destroy. */
CT_API ct_status ct_plan(const ct_desc *desc, ct_plan_t **out);

/* Name of the kernel the plan runs ("generic", "dense_tc", ...).  The string
 * is static; NULL plan gives "". */
CT_API const char *ct_plan_kernel(const ct_plan_t *plan);

/* Number of kernels one ct_run of this plan launches (for launch accounting). */
CT_API ct_status ct_plan_launches(const ct_plan_t *plan, int32_t *launches);

/* Bytes of device memory the caller provides for the pre-packed weight. */
CT_API ct_status ct_prepacked_weight_bytes(const ct_plan_t *plan, size_t *bytes);

/* Bytes of device scratch ct_run needs (0 when the kernel needs none). */
CT_API ct_status ct_workspace_bytes(const ct_plan_t *plan, size_t *bytes);

/* Re-lay W (the declared layout, device memory) into the plan's packed form
 * in w_packed (ct_prepacked_weight_bytes bytes, 16-byte aligned): taps split
 * into stride phases, tap order reversed within a phase, the reduction axis
 * contiguous (ai.onnx.ConvTranspose README, "Files": the 2-D/3-D weight
 * reorder templates).  Asynchronous on `stream` (a cudaStream_t, NULL for the
 * legacy default stream). */
CT_API ct_status ct_prepack_weights(const ct_plan_t *plan, const void *w, void *w_packed,
                             void *stream);

/* Y = ConvTranspose(X, W, B).  x, w_packed, bias (NULL when bias_len == 0),
 * y and workspace are device pointers; y is fully overwritten, including
 * positions no tap reaches, which receive the bias (or zero).  Asynchronous
 * on `stream`; a launch error returns CT_ERR_DEVICE. */
CT_API ct_status ct_run(const ct_plan_t *plan, const void *x, const void *w_packed,
                 const void *bias, void *y, void *workspace, void *stream);

/* Parts of one ct_run, for measuring them apart (ct_run_parts).  A call
 * consists of preparation launches (the re-layout of X into the workspace,
 * and the bias fill of outputs no tap reaches) followed by one main kernel
 * (the phase GEMM or gather).  Plans whose call is a single kernel have no
 * preparation: CT_PART_PREPARE alone launches nothing for them. */
#define CT_PART_PREPARE 1
#define CT_PART_MAIN 2
#define CT_PART_ALL 3

/* ct_run restricted to the parts in `parts` (a mask of CT_PART_*; 0 does
 * nothing, other bits are CT_ERR_ATTR).  ct_run(...) is ct_run_parts(...,
 * CT_PART_ALL).  CT_PART_MAIN alone reads the workspace and Y as an earlier
 * CT_PART_PREPARE call with the same x, workspace and y left them: a
 * benchmark prepares once and then times the main kernel by itself.  With
 * anything else in the workspace the main kernel still reads and writes
 * only inside the planned buffers, but Y is not the operator's result.
 * Arguments, alignment and errors as for ct_run. */
CT_API ct_status ct_run_parts(const ct_plan_t *plan, const void *x, const void *w_packed,
                              const void *bias, void *y, void *workspace, void *stream,
                              int32_t parts);

/* Size of the device array that ct_run_noalloc uses as its workspace.  Every
 * GPU that loads libct.so holds this much device memory until the process
 * exits. */
#define CT_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/* ct_run for callers that cannot allocate device memory while running, such
 * as a plugin inside an engine that owns all device memory, or a loop whose
 * rules forbid allocation after start-up.  The ONNX page and the ClikaRT page
 * have no counterpart of this call; it exists only for such callers.  The
 * caller still passes x, w_packed, bias and y as for ct_run.  The workspace
 * comes from a fixed array of CT_NOALLOC_SCRATCH_BYTES inside the library:
 * plans whose ct_workspace_bytes exceed that return CT_ERR_WORKSPACE.  Every
 * call looks up the array's device address on the current device
 * (cudaGetSymbolAddress; host code only ever sees a stand-in for the array,
 * never its device address).  With CUDA's lazy module loading the first such
 * lookup on a device loads the module that holds the array, which takes
 * CT_NOALLOC_SCRATCH_BYTES of device memory at that moment: make the first
 * call on each device at start-up, before any stream capture and before the
 * caller hands the rest of the device memory to its own allocator.  Later
 * calls allocate nothing.  All calls share the one array (it keeps the last
 * call's contents; the kernels overwrite all workspace bytes they read), so
 * calls whose GPU work overlaps in time, for example on two streams, race on
 * it and must be serialised by the caller. */
CT_API ct_status ct_run_noalloc(const ct_plan_t *plan, const void *x, const void *w_packed,
                                const void *bias, void *y, void *stream);

CT_API void ct_plan_destroy(ct_plan_t *plan);

/* ---- the operators that follow a transposed convolution in a decoder -------
 *
 * Dropout.  Element i of a tensor (its row-major index) is kept when a 16-bit
 * random value is at least t = floor(65536 p + 1/2), and then scaled by
 * 65536 / (65536 - t), so that the expectation is the input whatever p is;
 * it is 0 otherwise, also where the input is infinite or NaN.  p is in
 * [0, 1] and takes effect as t / 65536.  The value is 16-bit part i % 8 (low
 * half of word 0 first) of Philox4x32-10 (Salmon et al., "Parallel random
 * numbers: as easy as 1, 2, 3", 2011) with the four counter words (i / 8 low,
 * i / 8 high, offset low, offset high) and the key (seed low, seed high).
 * The mask is thus a function of (i, seed, offset): it is never stored, and
 * the gradient draws it again.  `rng`, when not NULL, points to two 64-bit
 * words on the device (8-byte aligned), seed and offset, which the kernel
 * reads in place of the arguments: a captured graph can so draw another mask
 * at each replay.  A step uses a new offset for each step and a new seed, or
 * an offset of its own, for each tensor. */

/* y = drop(x) + residual, computed in fp32 and rounded once.  n elements;
 * residual may be NULL.  y may be x or residual; other overlap, with the words
 * at rng too, is not allowed.  The gradient in x is this call on dy with the
 * same p, seed and offset and no residual; the gradient in the residual is dy
 * itself. */
CT_API ct_status ct_dropout(int32_t dtype, int64_t n, const void *x, const void *residual, double p,
                            uint64_t seed, uint64_t offset, const void *rng, void *y, void *stream);

/* Group norm of channels-last images x[N, S, C] (S pixels, of any number of
 * axes), C / groups neighbouring channels to a group, followed by an
 * activation and dropout:
 *
 *     mean = sum x / M,  rstd = (sum (x - mean)^2 / M + eps)^-1/2   per (image, group),
 *     a = (x - mean) * rstd * weight[c] + bias[c],   y = drop(act(a)),
 *
 * with M = S * C / groups.  Everything is computed in fp32 and y rounded
 * once.  dtype is x's, y's, dy's and dx's; param_dtype weight's, bias's and
 * their gradients', CT_F32 or dtype.  Limits: N <= 2^30, 1 <= C <= 2^24,
 * N * S * C <= 2^60 (CT_ERR_CHANNELS for C and groups, else CT_ERR_ATTR). */
typedef struct ct_group_norm_desc {
    int32_t dtype;         /* ct_dtype */
    int32_t param_dtype;   /* CT_F32, or dtype */
    int32_t activation;    /* ct_activation */
    int32_t reserved;      /* not read */
    int64_t N, S, C, groups;
    double eps;            /* >= 0 */
} ct_group_norm_desc;

/* Bytes of device workspace (256-byte aligned) of one forward and one
 * backward call; 0 where small images need none, the workspace pointer may
 * then be NULL.  Its contents need not be set before a call and mean
 * nothing after it; calls that may run at the same time need one each. */
CT_API ct_status ct_group_norm_workspace_bytes(const ct_group_norm_desc *desc, size_t *forward_bytes,
                                               size_t *backward_bytes);

/* Forward.  weight and bias may be NULL (1 and 0).  mean and rstd, each
 * [N, groups] fp32, may be NULL; the backward call needs them.  p = 0: no
 * dropout, seed, offset and rng are then not read.  Asynchronous on `stream`.
 * y, mean and rstd may overlap neither each other nor anything that the call
 * reads: x, weight, bias and the words at rng. */
CT_API ct_status ct_group_norm(const ct_group_norm_desc *desc, const void *x, const void *weight,
                               const void *bias, double p, uint64_t seed, uint64_t offset, const void *rng,
                               void *y, float *mean, float *rstd, void *workspace, void *stream);

/* Backward: dx (of x), dweight and dbias (of weight and bias, summed over
 * images and pixels), each NULL when it is not wanted.  x, weight, bias,
 * mean, rstd, p, seed, offset and rng as the forward call had and gave them;
 * a is computed again from x.  With S or N of 0 the parameters' gradients
 * are 0, and the other tensors are not read and may be NULL.  dx, dweight and
 * dbias may overlap neither each other nor anything that the call reads.  The
 * same call gives the same bits: no sum's order depends on timing. */
CT_API ct_status ct_group_norm_backward(const ct_group_norm_desc *desc, const void *dy, const void *x,
                                        const float *mean, const float *rstd, const void *weight,
                                        const void *bias, double p, uint64_t seed, uint64_t offset,
                                        const void *rng, void *dx, void *dweight, void *dbias,
                                        void *workspace, void *stream);

/* Root-mean-square norm of `rows` rows of C channels (pixels, tokens or heads,
 * dense), of x or of x plus a residual:
 *
 *     h = x + residual,   rstd = (sum_c h^2 / C + eps)^-1/2,   y[c] = h[c] * rstd * weight[c].
 *
 * h is formed in fp32; `sum` gets it rounded to dtype (what the residual
 * stream carries on), y and rstd come from the unrounded values.  Everything
 * is computed in fp32 and rounded once; the squares' sum too: a row whose 2-norm
 * passes 1.8e19 (a root mean square of 1.8e19 / sqrt(C)) has an rstd of 0.
 * dtype is x's, residual's, y's and sum's; param_dtype weight's and its
 * gradient's, CT_F32 or dtype.
 *
 * e4m3 output: y is not rounded to dtype but held as codes and fp32 scales,
 *     scale = max(max |y| * (1 / 448), 2^-126) of a block,   q = e4m3(y * (1 / scale)), to nearest even,
 * each reciprocal and product rounded to fp32;
 * a block is `block` neighbouring channels of a row (32, 64 or 128; the last
 * one of a row may be shorter), or all C of them for 0.  q * scale is the
 * value.  A block with a NaN or an infinity in it (of y: a weight can make one
 * of a finite h) has a scale of NaN.
 *
 * Limits: 1 <= C <= 2^24 (CT_ERR_CHANNELS), rows * C <= 2^60. */
typedef struct ct_rms_norm_desc {
    int32_t dtype;         /* ct_dtype */
    int32_t param_dtype;   /* CT_F32, or dtype */
    int32_t block;         /* channels under one scale, 0: all of a row.  ct_rms_norm_e4m3 alone reads it */
    int32_t reserved;      /* not read */
    int64_t rows, C;
    double eps;            /* >= 0 */
} ct_rms_norm_desc;

/* Bytes of device workspace (256-byte aligned) of a backward call that wants
 * dweight; the forward calls need none.  Its contents need not be set before
 * a call and mean nothing after it; calls that may run at the same time need
 * one each. */
CT_API ct_status ct_rms_norm_workspace_bytes(const ct_rms_norm_desc *desc, size_t *backward_bytes);

/* Forward.  residual, weight (1), sum and rstd ([rows] fp32) may be NULL; sum
 * needs a residual.  y may be x or residual, and sum too, each exactly; else
 * no output may overlap another one or anything that the call reads.
 * Asynchronous on `stream`. */
CT_API ct_status ct_rms_norm(const ct_rms_norm_desc *desc, const void *x, const void *residual, const void *weight,
                             void *y, void *sum, float *rstd, void *stream);

/* Forward with e4m3 output: q [rows, C] (one byte each), scale [rows] or, with
 * a block, [rows, ceil(C / block)].  The rest as ct_rms_norm; q and scale may
 * overlap nothing that the call reads. */
CT_API ct_status ct_rms_norm_e4m3(const ct_rms_norm_desc *desc, const void *x, const void *residual,
                                  const void *weight, void *q, float *scale, void *sum, float *rstd, void *stream);

/* Backward: dx, the gradient in x and in the residual alike, and dweight,
 * summed over the rows; each NULL when it is not wanted.  x is what was normed
 * (sum where there was a residual), rstd as the forward call gave it; dsum,
 * the gradient that reaches `sum` on its own way, is added to dx and may be
 * NULL.  With rows of 0 dweight is 0 and the other tensors are not read.
 * Outputs may overlap neither each other nor anything that the call reads.
 * The same call gives the same bits. */
CT_API ct_status ct_rms_norm_backward(const ct_rms_norm_desc *desc, const void *dy, const void *x, const float *rstd,
                                      const void *weight, const void *dsum, void *dx, void *dweight,
                                      void *workspace, void *stream);

/* Rotary positions of channels-last heads x[N, S, heads, dim], S pixels on 1
 * to 3 axes.  Of each head the first sum(sections) elements are rotated in
 * pairs, sections[a] of them (an even number) by the position on axis a; the
 * rest stay as they are.  Pair i (of the first sum(sections) / 2, those of
 * axis 0 first) is elements 2i and 2i + 1 (CT_PAIRS_ADJACENT) or i and
 * i + sum(sections) / 2 (CT_PAIRS_HALVES); the j-th pair of axis a turns by
 *
 *     t = position * base^(-2 j / sections[a]),   (u, v) -> (u cos t - v sin t, u sin t + v cos t).
 *
 * The frequency is rounded to 64 bits, for positions up to 2^24 (and 2^22
 * turns) then to two floats of 48 bits together; their product with the position
 * is formed in two floats, beyond that in 64 bits (one that those do not hold is
 * no angle, and gives NaN).  Cosine and sine are fp32, off by at most 1.5 * 2^-24
 * plus 2^-45 of the angle (2^-51 in 64 bits); the rotation
 * is fp32, rounded once.  The gradient in x is the inverse rotation of dy
 * (`inverse`: by -t). */
typedef enum ct_pairs { CT_PAIRS_ADJACENT = 0, CT_PAIRS_HALVES = 1 } ct_pairs;

/* Positions: the pixels' indices on the grid, or numbers [S, axes] on the
 * device, one such array for every image or one for all. */
typedef enum ct_position_type {
    CT_POSITION_GRID = 0,
    CT_POSITION_I32 = 1,
    CT_POSITION_I64 = 2,
    CT_POSITION_F32 = 3
} ct_position_type;

/* Strides are in elements, a head's own elements are neighbours.  x may
 * repeat (strides of 0); y's elements must be apart.  Limits: N, heads, dim
 * and the grid's sizes in [0, 2^30], dim >= 1, sum(sections) <= dim and <=
 * 512, each section >= 0 and even (CT_ERR_CHANNELS), 1 to 3 axes
 * (CT_ERR_SPAN), base > 0 and finite, every frequency finite in 64 bits (bases
 * from 2^-1022 on are), at most 2^60 elements, and no stride past 2^60 / 4 in
 * magnitude; y's not negative (CT_ERR_ATTR). */
typedef struct ct_rotary_desc {
    int32_t dtype;          /* ct_dtype */
    int32_t axes;           /* 1..3 */
    int32_t pairs;          /* ct_pairs */
    int32_t inverse;        /* 0, or 1: rotate by -t */
    int32_t position_type;  /* ct_position_type */
    int32_t position_images;/* 1: positions [N, S, axes]; 0: [S, axes] for every image */
    int64_t N;
    int64_t grid[3];        /* pixels along each axis, S their product (given positions too) */
    int64_t heads, dim;
    int64_t sections[3];
    int64_t x_strides[3];   /* image, pixel, head */
    int64_t y_strides[3];
    double base;
} ct_rotary_desc;

/* y = rotated x.  y may be x with the same strides, else it may overlap
 * nothing that the call reads.  positions is NULL for CT_POSITION_GRID.
 * Asynchronous on `stream`. */
CT_API ct_status ct_rotary(const ct_rotary_desc *desc, const void *x, const void *positions, void *y, void *stream);

/* AdamW over many tensors at once (Loshchilov and Hutter, "Decoupled weight
 * decay regularization", 2019).  For every element, in fp32:
 *
 *     g' = g * grad_scale,   m = beta1 m + (1 - beta1) g',   v = beta2 v + (1 - beta2) g'^2,
 *     p  = p - lr (weight_decay p + m / (1 - beta1^step) / (sqrt(v / (1 - beta2^step)) + eps)).
 *
 * Parameters and gradients are dense tensors of their own; the states of all
 * parameters lie in one buffer for each kind, parameter i's from block
 * sum_{k < i} ceil(n_k / 256) on, a block being 256 elements (what a parameter
 * leaves of its last block counts for nothing; updates set it to 0).
 * Parameters of 16 bits have a master in fp32 that the update works on, in a
 * buffer of blocks for them alone; the parameter is the master rounded.
 *
 * bits = 32: exp_avg (m) and exp_avg_sq (v) are fp32.  bits = 8: they are e4m3
 * codes with one fp32 scale a block (exp_avg_scale, exp_avg_sq_scale), of m
 * and of the square root of v; scale = max(max / 448, 2^-126), and a value is
 * rounded up to the next code with the probability of the part that lies beyond
 * the last (nearest rounding would drop every change below half a step).  The
 * random number is 16-bit part i % 8 of Philox4x32-10 (as in dropout) at
 * (i / 8, step) under the key `seed`, i the element's place in the states.  A
 * positive root never becomes 0.  A gradient that is not finite, or past
 * 1.8e19 (its square is not), makes its element not finite, with 8-bit states
 * its block; v below 2^-126 has a smaller root than it should. */
typedef struct ct_param {
    int64_t n;              /* elements */
    int32_t dtype;          /* ct_dtype of the parameter */
    int32_t grad_dtype;     /* of its gradient: dtype or CT_F32 */
    double weight_decay;    /* >= 0, within fp32; read by ct_adamw alone */
} ct_param;

typedef struct ct_adamw_desc {
    int32_t bits;           /* 32 or 8 */
    int32_t reserved;       /* not read */
    double lr, beta1, beta2, eps;   /* lr >= 0, betas in [0, 1), eps >= 2^-126; fp32 holds them (CT_ERR_ATTR) */
    int64_t step;           /* 1 for the first update */
    uint64_t seed;          /* bits = 8 alone */
    /* on the device, read by the kernel in place of the numbers above; NULL:
     * not.  A captured graph so takes another step and rate at each replay.
     * A rate that is negative or not finite, a step below 1 and a grad_scale
     * that is no positive finite number skip the update: nothing is written. */
    const float *lr_device;
    const int64_t *step_device;
    const float *grad_scale;    /* NULL: 1 */
} ct_adamw_desc;

/* One update.  shapes, params and grads are host arrays of `count` entries, read
 * before the call returns; a NULL gradient leaves its parameter and states as
 * they are.  params[i] (and grads[i]) may not overlap each other or anything
 * else of the call.  master may be NULL without parameters of 16 bits, the
 * scales with bits = 32; states, masters and scales are 256-byte aligned.
 * Limits: count <= 2^20, at most 2^40 elements (CT_ERR_ATTR).  Asynchronous on
 * `stream`, a launch for up to 512 tensors. */
CT_API ct_status ct_adamw(const ct_adamw_desc *desc, int64_t count, const ct_param *shapes, void *const *params,
                          const void *const *grads, void *exp_avg, void *exp_avg_sq, float *exp_avg_scale,
                          float *exp_avg_sq_scale, float *master, void *stream);

/* *norm = the square root of the sum of all gradients' squares, to its rounding
 * (squares and sums in 64 bits; those of 16-bit gradients, exact in fp32, in
 * sums of two floats, 48 bits, for up to 32 of them), *scale (may be NULL) =
 * min(1, max_norm / norm), or 0 where the norm is not finite in fp32: what
 * ct_adamw's grad_scale takes to clip, or to skip an update that overflowed.
 * Of shapes, n and grad_dtype are read; a NULL gradient counts nothing.
 * max_norm > 0, infinity allowed.  The same call gives the same bits. */
CT_API ct_status ct_grad_norm_workspace_bytes(int64_t count, size_t *bytes);
CT_API ct_status ct_grad_norm(int64_t count, const ct_param *shapes, const void *const *grads, double max_norm,
                              float *norm, float *scale, void *workspace, void *stream);

/* Static, human-readable text for a status code. */
CT_API const char *ct_status_string(ct_status status);

/* Failure report of the kernels' bounded waits.  Every wait of the
 * tensor-core and grouped kernels on an mbarrier gives up after about one
 * second of SM clock; the kernel then records a code in its module's device
 * error word, skips the rest of its work (so Y is not valid) and returns, and
 * the device stays usable.  This call waits for `stream` (work that ran
 * earlier on other streams must be finished by the caller), then reads and
 * clears the error words of the current device.  *code = 0 and CT_OK when no
 * wait ran out since the last call; otherwise *code = 100 * module + wait
 * site (module 1 dense_tc, 2 dense_tc_pair, 3 dense_tc_pertap, 4 grouped,
 * 5 the self-test below) and CT_ERR_DEVICE.  CT_ERR_DEVICE with *code = 0
 * means a CUDA call failed (or the current device is not an sm_100 part). */
CT_API ct_status ct_take_device_error(void *stream, int32_t *code);

/* Self-test of the bounded-wait failure path (no counterpart on the pages).
 * One block of one thread runs the steps every tensor-core kernel takes when
 * a wait runs out: it starts a bulk copy of 4 KB into its shared memory,
 * then waits, with a limit of `limit_cycles` SM clock cycles (1 .. 2^31),
 * on an mbarrier that nothing ever arrives at.  When the limit runs out it
 * records wait site 1 in module 5's error word, waits (with the kernels'
 * usual one-second limit) for its copy still in flight, and returns.  So
 * after a call, ct_take_device_error reports code 501 and the device stays
 * usable; site 2 would mean the copy never completed.  Asynchronous on
 * `stream`; CT_ERR_ATTR for a limit outside the range. */
CT_API ct_status ct_selftest_wait_timeout(void *stream, int64_t limit_cycles);

#ifdef __cplusplus
}
#endif

#endif /* CT_H_ */
