#include "rms_norm_kernels.cuh"

namespace ct {

ct_status rms_forward_bf16(const RmsArgs &a, const RmsGeom &g, cudaStream_t st) {
    return forward_t<__nv_bfloat16>(a, g, st);
}
ct_status rms_backward_bf16(const RmsArgs &a, const RmsGeom &g, cudaStream_t st) {
    return backward_t<__nv_bfloat16>(a, g, st);
}

}  // namespace ct
