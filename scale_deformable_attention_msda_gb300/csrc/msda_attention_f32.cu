#include "msda_attention_simple.cuh"

namespace msda {
cudaError_t launch_attention_f32(int mode, const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    return launch_simple(mode, a, blocks, stream);
}
}  // namespace msda
