// Layer norm's backward kernels for fp32 and fp64 data (a unit of its own, so that the types
// compile side by side).
#include "msda_norm_backward.cuh"

namespace msda {

cudaError_t launch_norm_backward_f32(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    return launch_backward_t<float, float>(a, p, stream);
}
cudaError_t launch_norm_backward_f64(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    return launch_general<double, double>(a, p, stream);
}

}  // namespace msda
