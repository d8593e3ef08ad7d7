// The group norm's kernels for fp16 tensors.
#include "group_norm_kernels.cuh"

namespace ct {

ct_status gn_forward_f16(const GnGeom &g, const GnArgs &a, cudaStream_t st) { return forward_t<__half>(g, a, st); }
ct_status gn_backward_f16(const GnGeom &g, const GnArgs &a, cudaStream_t st) { return backward_t<__half>(g, a, st); }

}  // namespace ct
