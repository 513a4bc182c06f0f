// Attention's small kernels: the mask packed to bits, the backward's row sums
// dO out, and the join of split columns.
#include "msda_attention_host.h"

namespace msda {
namespace {

constexpr int kPackQ = 64, kPackK = 128;

// Bits of a tile of 64 queries by 128 keys: read once in bytes, written as words
// along the keys (by_query), as words along the queries (by_key; NULL: not
// wanted), and as the class of each granule of 64 by 64. Each head and mode
// reads the bits, so that a mask shared by 8 heads is read in bytes once and
// otherwise costs an eighth. Q = 1 (a row that serves all queries): by_key has a
// word of ones or zeros for each key.
__global__ void __launch_bounds__(256) attn_pack_kernel(const AttnMaskSource m, uint32_t *by_query, int words_q,
                                                        uint32_t *by_key, int words_k, uint8_t *classes, int granules) {
    __shared__ uint32_t word[kPackQ][kPackK / 32 + 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int tk = granules / 2, tq = (m.Q + kPackQ - 1) / kPackQ;
    int64_t t = blockIdx.x;
    const int k0 = (int)(t % tk) * kPackK;
    t /= tk;
    const int q0 = (int)(t % tq) * kPackQ;
    const int64_t bh = t / tq;
    const int b = (int)(bh / m.M), h = (int)(bh % m.M);
    const uint8_t *from = m.p + b * m.batch + h * m.head;
#pragma unroll 8
    for (int i = 0; i < kPackQ * (kPackK / 32) / 8; ++i) {
        const int r = warp + 8 * (i / (kPackK / 32)), c = i % (kPackK / 32);
        const int q = q0 + r, k = k0 + 32 * c + lane;
        const bool on = q < m.Q && k < m.S && from[q * m.query + k * m.key] != 0;
        const uint32_t bits = __ballot_sync(0xffffffffu, on);
        if (lane == c) word[r][c] = bits;
    }
    __syncthreads();
    const int rows = min(kPackQ, m.Q - q0);
    for (int i = threadIdx.x; i < rows * (kPackK / 32); i += 256) {
        const int r = i / (kPackK / 32), c = i % (kPackK / 32);
        by_query[(bh * m.Q + q0 + r) * words_q + k0 / 32 + c] = word[r][c];
    }
    if (warp < 2) {                    // two granules of keys
        uint32_t any = 0u, all = 0xffffffffu;
        for (int r = lane; r < rows; r += 32) {
            any |= word[r][2 * warp] | word[r][2 * warp + 1];
            all &= word[r][2 * warp] & word[r][2 * warp + 1];
        }
        any = __reduce_or_sync(0xffffffffu, any);
        all = __reduce_and_sync(0xffffffffu, all);
        if (lane == 0) classes[(bh * tq + q0 / kPackQ) * granules + k0 / kAttnGranule + warp] = !any ? 0 : ~all ? 1 : 2;
    }
    if (by_key) {                      // 8 warps: 4 words of keys by 2 words of queries
        const int c = warp % 4, half = warp / 4;
        const uint32_t mine = word[32 * half + lane][c];
        uint32_t turned = 0u;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t bits = __ballot_sync(0xffffffffu, (mine >> i) & 1u);
            if (lane == i) turned = bits;
        }
        const int k = k0 + 32 * c + lane;
        if (k < m.S) {
            if (m.Q > 1) by_key[(bh * m.S + k) * words_k + q0 / 32 + half] = turned;
            else if (half == 0) by_key[bh * m.S + k] = turned ? 0xffffffffu : 0u;
        }
    }
}

constexpr int kDeltaThreads = 512, kDeltaBlocks = 304;

// The queries' stat: the row sums delta = sum over channels of dO out, L lanes a row
// of 16 bytes each, beside the forward's lse. fp16 (norm_do given): also the largest
// finite |dO_i|^2 and |v_j|^2 of what this block has seen.
template <typename T, int L>
__global__ void __launch_bounds__(kDeltaThreads) attn_delta_kernel(const AttnArgs a) {
    constexpr int V = 16 / sizeof(T), per = kDeltaThreads / L;
    const int lane = threadIdx.x % L, d = lane * V;
    const int64_t rows = (int64_t)a.B * a.stat_row * a.M;
    float most_do = 0.0f, most_v = 0.0f;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < rows; r0 += (int64_t)gridDim.x * per) {
        const int64_t r = r0 + threadIdx.x / L, bq = r / a.M;
        const int m = (int)(r % a.M), b = (int)(bq / a.stat_row), q = (int)(bq % a.stat_row);
        const bool valid = r < rows && q < a.Q;
        float dot = 0.0f, square = 0.0f;
        if (valid && d < a.D) {
            const int64_t at = (((int64_t)b * a.Q + q) * a.M + m) * a.D + d;
            float x[V], y[V];
            unpack16<T>(x, ldg16(static_cast<const T *>(a.go.p) + at));
            unpack16<T>(y, ldg16(static_cast<const T *>(a.o.p) + at));
            if (a.rest) {
                float z[V];
                unpack16<T>(z, ldg16(static_cast<const T *>(a.rest) + at));
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] += z[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dot = fmaf(x[i], y[i], dot);
                square = fmaf(x[i], x[i], square);
            }
        }
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) {
            dot += __shfl_xor_sync(0xffffffffu, dot, off);
            square += __shfl_xor_sync(0xffffffffu, square, off);
        }
        if (isfinite(square)) most_do = fmaxf(most_do, square);
        if (r < rows && lane == 0) {
            float *to = attn_stat(a, b, m, q);
            to[0] = valid ? a.up - attn_lse2(a.lse[((int64_t)b * a.M + m) * a.Q + q]) : -INFINITY;
            to[2] = valid ? -dot : 0.0f;
        }
    }
    if (!a.norm_do) return;
    const int64_t keys = (int64_t)a.B * a.S * a.N;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < keys; r0 += (int64_t)gridDim.x * per) {
        const int64_t r = r0 + threadIdx.x / L;
        float square = 0.0f;
        if (r < keys && d < a.D) {
            const int64_t bs = r / a.N;
            float x[V];
            unpack16<T>(x, ldg16(attn_at<T>(a.v, (int)(bs / a.S), (int)(bs % a.S), (int)(r % a.N)) + d));
#pragma unroll
            for (int i = 0; i < V; ++i) square = fmaf(x[i], x[i], square);
        }
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) square += __shfl_xor_sync(0xffffffffu, square, off);
        if (isfinite(square)) most_v = fmaxf(most_v, square);
    }
    __shared__ float part[2][kDeltaThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        most_do = fmaxf(most_do, __shfl_xor_sync(0xffffffffu, most_do, off));
        most_v = fmaxf(most_v, __shfl_xor_sync(0xffffffffu, most_v, off));
    }
    if (threadIdx.x % 32 == 0) {
        part[0][threadIdx.x / 32] = most_do;
        part[1][threadIdx.x / 32] = most_v;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        float most = 0.0f;
        for (int i = 0; i < kDeltaThreads / 32; ++i) most = fmaxf(most, part[threadIdx.x][i]);
        (threadIdx.x ? a.norm_v : a.norm_do)[blockIdx.x] = most;
    }
}

template <typename T> cudaError_t launch_delta(const AttnArgs &a, cudaStream_t stream) {
    const int lanes = a.D * (int)sizeof(T) / 16;
    if (lanes <= 4) attn_delta_kernel<T, 4><<<a.norms, kDeltaThreads, 0, stream>>>(a);
    else if (lanes <= 8) attn_delta_kernel<T, 8><<<a.norms, kDeltaThreads, 0, stream>>>(a);
    else if (lanes <= 16) attn_delta_kernel<T, 16><<<a.norms, kDeltaThreads, 0, stream>>>(a);
    else attn_delta_kernel<T, 32><<<a.norms, kDeltaThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

// Sums of the splits, four channels a thread. Forward: each split's sums are
// relative to its own maximum, and its weight is exp2 of the distance.
template <typename T>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a, int mode) {
    const int per = a.D / 4;
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x, row = i / per;
    const int d = (int)(i % per) * 4;
    if (row >= a.part_rows) return;
    const int64_t step = a.part_rows * a.D;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (mode == kForward) {
        const float *ml = a.part + a.splits * step + 2 * row;
        float top = -INFINITY, sum = 0.0f;
        for (int s = 0; s < a.splits; ++s) top = fmaxf(top, ml[2 * s * a.part_rows]);
        const float base = top == -INFINITY ? 0.0f : top;
        for (int s = 0; s < a.splits; ++s) {
            const float f = exp2f(ml[2 * s * a.part_rows] - base);
            const float4 v = *reinterpret_cast<const float4 *>(a.part + s * step + row * a.D + d);
            sum = fmaf(f, ml[2 * s * a.part_rows + 1], sum);
            acc = make_float4(fmaf(f, v.x, acc.x), fmaf(f, v.y, acc.y), fmaf(f, v.z, acc.z), fmaf(f, v.w, acc.w));
        }
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float v[4] = {acc.x * f, acc.y * f, acc.z * f, acc.w * f};
#pragma unroll
        for (int k = 0; k < 4; ++k) attn_put<T>(a.out, a.rest, row * a.D + d + k, v[k]);
        if (a.lse && d == 0) {
            const int m = (int)(row % a.M);
            const int64_t bq = row / a.M;
            a.lse[(bq / a.Q * a.M + m) * a.Q + bq % a.Q] = sum == 0.0f ? -INFINITY : (base + log2f(sum)) * kLn2;
        }
        return;
    }
    for (int which = 0; which < (mode == kGradKV ? 2 : 1); ++which) {
        acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s = 0; s < a.splits; ++s) {
            const float4 v = *reinterpret_cast<const float4 *>(a.part + (which * a.splits + s) * step + row * a.D + d);
            acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
        }
        const float f = mode == kGradQ || which ? a.scale : 1.0f;
        T *to = static_cast<T *>(mode == kGradQ ? a.gq : which ? a.gk : a.gv) + row * a.D + d;
        to[0] = Elem<T>::from_f(acc.x * f);
        to[1] = Elem<T>::from_f(acc.y * f);
        to[2] = Elem<T>::from_f(acc.z * f);
        to[3] = Elem<T>::from_f(acc.w * f);
    }
}

}  // namespace

cudaError_t launch_attention_pack(const AttnMaskSource &m, uint32_t *by_query, int words_q, uint32_t *by_key,
                                  int words_k, uint8_t *classes, int granules, cudaStream_t stream) {
    const int64_t blocks = (int64_t)m.B * m.M * ((m.Q + kPackQ - 1) / kPackQ) * (granules / 2);
    attn_pack_kernel<<<(unsigned)blocks, 256, 0, stream>>>(m, by_query, words_q, by_key, words_k, classes, granules);
    return cudaGetLastError();
}

cudaError_t launch_attention_delta(const AttnArgs &a, msda_dtype_t dt, cudaStream_t stream) {
    return dt == MSDA_F32 ? launch_delta<float>(a, stream)
         : dt == MSDA_BF16 ? launch_delta<__nv_bfloat16>(a, stream) : launch_delta<__half>(a, stream);
}

cudaError_t launch_attention_join(int mode, const AttnArgs &a, msda_dtype_t dt, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((a.part_rows * (a.D / 4) + 127) / 128);
    if (dt == MSDA_F32) attn_join_kernel<float><<<blocks, 128, 0, stream>>>(a, mode);
    else if (dt == MSDA_BF16) attn_join_kernel<__nv_bfloat16><<<blocks, 128, 0, stream>>>(a, mode);
    else attn_join_kernel<__half><<<blocks, 128, 0, stream>>>(a, mode);
    return cudaGetLastError();
}

}  // namespace msda
