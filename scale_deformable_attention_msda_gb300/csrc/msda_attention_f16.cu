#include "msda_attention_tc.cuh"

namespace msda {
cudaError_t launch_attention_f16(const AttnArgs &a, int64_t blocks, cudaStream_t stream) { return launch_tc<__half>(a, blocks, stream); }
cudaError_t launch_attention_f16_back(const AttnArgs &q, int64_t q_blocks, const AttnArgs &kv, int64_t kv_blocks, cudaStream_t stream) {
    return launch_tc_back<__half>(q, q_blocks, kv, kv_blocks, stream);
}
}  // namespace msda
