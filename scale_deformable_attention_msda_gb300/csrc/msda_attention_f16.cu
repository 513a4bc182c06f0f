#include "msda_attention_tc.cuh"

namespace msda {
cudaError_t launch_attention_f16(int mode, const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    return launch_tc<__half>(mode, a, blocks, stream);
}
}  // namespace msda
