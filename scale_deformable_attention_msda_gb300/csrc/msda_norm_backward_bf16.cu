// Layer norm's backward kernels for bf16 data (a unit of its own, so that the types
// compile side by side).
#include "msda_norm_backward.cuh"

namespace msda {

// wide: fp32 parameters.
cudaError_t launch_norm_backward_bf16(const NormArgs &a, const NormPlan &p, bool wide, cudaStream_t stream) {
    return wide ? launch_backward_t<__nv_bfloat16, float>(a, p, stream) : launch_backward_t<__nv_bfloat16, __nv_bfloat16>(a, p, stream);
}

}  // namespace msda
