// Attention's launches, by type (host declarations).
#pragma once

#include <cuda_runtime.h>

#include "msda_attention.cuh"

namespace msda {

cudaError_t launch_attention_f32(int mode, const AttnArgs &a, int64_t blocks, cudaStream_t stream);
cudaError_t launch_attention_bf16(const AttnArgs &a, int64_t blocks, cudaStream_t stream);        // forward
cudaError_t launch_attention_f16(const AttnArgs &a, int64_t blocks, cudaStream_t stream);
cudaError_t launch_attention_bf16_back(const AttnArgs &q, int64_t q_blocks, const AttnArgs &kv, int64_t kv_blocks, cudaStream_t stream);
cudaError_t launch_attention_f16_back(const AttnArgs &q, int64_t q_blocks, const AttnArgs &kv, int64_t kv_blocks, cudaStream_t stream);

// A launch that may start while the kernel before it in the stream ends (chained; see
// attn_after).
template <class... P, class... A>
cudaError_t launch_after(bool chained, void (*kernel)(P...), int64_t blocks, int threads, size_t shared, cudaStream_t stream, const A &...args) {
    cudaLaunchAttribute attribute = {};
    attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attribute.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((unsigned)blocks);
    config.blockDim = dim3((unsigned)threads);
    config.dynamicSmemBytes = shared;
    config.stream = stream;
    config.attrs = &attribute;
    config.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&config, kernel, P(args)...);
}

// Whether a key tile's few queries are walked by small blocks, two an SM, one starting while
// the other ends, in a launch of their own, rather than by one an SM with tiles of 128 columns
// beside the queries' gradients. The whole backward, 4 x 8 heads of 32, bf16, small blocks and
// large: 120 queries over 2,400 keys 31.0 us, 38.8, over 1,200 (320 key tiles) 26.7 and 23.2,
// over 200 16.6 and 9.3; 300 queries over 300 keys 25.8 and 21.4.
constexpr bool tc_short(int mode, int64_t D, int64_t Q, int64_t G, int64_t key_tiles) {
    return mode == kGradKV && D <= 64 && G * ((Q + 63) / 64 * 64) <= 256 && key_tiles > 456;
}
inline bool tc_short(const AttnArgs &a) { return tc_short(kGradKV, a.D, a.Q, a.G, (int64_t)a.B * a.N * (((int64_t)a.S + 127) / 128)); }
// The 16-bit kernels' columns of a tile, and their blocks of an SM.
constexpr int tc_columns(int mode, int64_t D, bool is_short) { return is_short || (mode == kForward && D > 64) ? 64 : 128; }
constexpr int tc_blocks(int mode, int64_t D, bool is_short) { return is_short || mode == kForward ? 2 : 1; }

// The fp32 kernels' blocks of an SM, by registers and shared memory.
constexpr int simple_blocks(int64_t D) { return D <= 64 ? 2 : 1; }

// The forward in fp32 of at most four rows a key head (see msda_attention_few.cu).
constexpr bool few_rows(int mode, msda_dtype_t dt, int64_t Q, int64_t G) { return mode == kForward && dt == MSDA_F32 && Q * G <= 4; }
cudaError_t launch_attention_few(const AttnArgs &a, int64_t blocks, cudaStream_t stream);

// What the mask is made of before it is packed: bytes at strides.
struct AttnMaskSource {
    const uint8_t *p;
    int64_t batch, head, query, key;
    int B, M, Q, S;                    // Q is 1 where one row serves all queries
};
cudaError_t launch_attention_pack(const AttnMaskSource &m, uint32_t *by_query, int words_q, uint32_t *by_key,
                                  int words_k, uint8_t *classes, int granules, cudaStream_t stream);
cudaError_t launch_attention_delta(const AttnArgs &a, int64_t blocks, msda_dtype_t dt, cudaStream_t stream);
cudaError_t launch_attention_join(int mode, const AttnArgs &a, msda_dtype_t dt, cudaStream_t stream);

}  // namespace msda
