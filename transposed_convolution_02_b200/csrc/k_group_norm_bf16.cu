// The group norm's kernels for bf16 tensors.
#include "group_norm_kernels.cuh"

namespace ct {

ct_status gn_forward_bf16(const GnGeom &g, const GnArgs &a, cudaStream_t st) { return forward_t<__nv_bfloat16>(g, a, st); }
ct_status gn_backward_bf16(const GnGeom &g, const GnArgs &a, cudaStream_t st) { return backward_t<__nv_bfloat16>(g, a, st); }

}  // namespace ct
