// Layer norm's forward kernels for fp32 and fp64 data (a unit of its own, so that the types
// compile side by side).
#include "msda_norm_forward.cuh"

namespace msda {

cudaError_t launch_norm_forward_f32(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    return launch_forward_t<float, float>(a, p, stream);
}
cudaError_t launch_norm_forward_f64(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    return launch(norm_forward_general_kernel<double, double>, a, p, 0, stream);
}

}  // namespace msda
