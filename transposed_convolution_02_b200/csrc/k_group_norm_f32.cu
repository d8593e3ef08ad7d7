// The group norm's kernels for fp32 tensors.
#include "group_norm_kernels.cuh"

namespace ct {

ct_status gn_forward_f32(const GnGeom &g, const GnArgs &a, cudaStream_t st) { return forward_t<float>(g, a, st); }
ct_status gn_backward_f32(const GnGeom &g, const GnArgs &a, cudaStream_t st) { return backward_t<float>(g, a, st); }

}  // namespace ct
