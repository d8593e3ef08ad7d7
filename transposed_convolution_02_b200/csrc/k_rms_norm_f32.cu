#include "rms_norm_kernels.cuh"

namespace ct {

ct_status rms_forward_f32(const RmsArgs &a, const RmsGeom &g, cudaStream_t st) { return forward_t<float>(a, g, st); }
ct_status rms_backward_f32(const RmsArgs &a, const RmsGeom &g, cudaStream_t st) { return backward_t<float>(a, g, st); }

}  // namespace ct
