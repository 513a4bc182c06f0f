// Attention's launches, by type (host declarations).
#pragma once

#include <cuda_runtime.h>

#include "msda_attention.cuh"

namespace msda {

cudaError_t launch_attention_f32(int mode, const AttnArgs &a, int64_t blocks, cudaStream_t stream);
cudaError_t launch_attention_bf16(int mode, const AttnArgs &a, int64_t blocks, cudaStream_t stream);
cudaError_t launch_attention_f16(int mode, const AttnArgs &a, int64_t blocks, cudaStream_t stream);

// The 16-bit kernels' columns of a tile, and their blocks of an SM.
constexpr int tc_columns(int mode, int D) { return mode == kForward && D > 64 ? 64 : 128; }
constexpr int tc_blocks(int mode, int D) { return mode != kForward ? 1 : 2; }

// What the mask is made of before it is packed: bytes at strides.
struct AttnMaskSource {
    const uint8_t *p;
    int64_t batch, head, query, key;
    int B, M, Q, S;                    // Q is 1 where one row serves all queries
};
cudaError_t launch_attention_pack(const AttnMaskSource &m, uint32_t *by_query, int words_q, uint32_t *by_key,
                                  int words_k, uint8_t *classes, int granules, cudaStream_t stream);
cudaError_t launch_attention_delta(const AttnArgs &a, msda_dtype_t dt, cudaStream_t stream);
cudaError_t launch_attention_join(int mode, const AttnArgs &a, msda_dtype_t dt, cudaStream_t stream);

}  // namespace msda
