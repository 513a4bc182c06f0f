// Attention's small kernels: the mask packed to bits, the backward's row sums
// dO out, and the join of split columns.
#include <type_traits>

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
    attn_after();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int tk = granules / 2, tq = (m.Q + kPackQ - 1) / kPackQ;
    int64_t t = blockIdx.x;
    const int k0 = (int)(t % tk) * kPackK;
    t /= tk;
    const int q0 = (int)(t % tq) * kPackQ;
    const int64_t bh = t / tq;
    const int b = (int)(bh / m.M), h = (int)(bh % m.M);
    const uint8_t *from = m.p + b * m.batch + h * m.head;
    constexpr int kWords = kPackQ * (kPackK / 32) / 8;     // of a warp; all its loads are under way at once
    uint8_t byte[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int q = q0 + warp + 8 * (i / (kPackK / 32)), k = k0 + 32 * (i % (kPackK / 32)) + lane;
        byte[i] = q < m.Q && k < m.S ? from[q * m.query + k * m.key] : 0;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const uint32_t bits = __ballot_sync(0xffffffffu, byte[i] != 0);
        if (lane == i % (kPackK / 32)) word[warp + 8 * (i / (kPackK / 32))][i % (kPackK / 32)] = bits;
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

constexpr int kDeltaThreads = 256;

// Which of the 32 keys from key0 on, a multiple of 32, some query of a key head attends: the
// class of the granule that they lie in, of 64 queries at a time, and where it is mixed each
// lane its key's bits. For a whole warp.
__device__ __forceinline__ uint32_t attn_attended(const AttnArgs &a, int b, int n, int key0) {
    const int key = key0 + (threadIdx.x & 31);
    uint32_t some = __ballot_sync(0xffffffffu, key < a.S);
    if (!a.classes) return some;
    const uint32_t there = some;
    some = 0u;
    for (int h = n * a.G; h < n * a.G + (a.class_head ? a.G : 1); ++h) {
        const uint8_t *c = a.classes + b * a.class_batch + h * a.class_head + key0 / kAttnGranule;
        const uint32_t *words = key < a.S ? attn_word_row<kGradKV>(a, b, h, key) : nullptr;
        for (int q = 0; q < (a.class_row ? a.Q : 1); q += kAttnGranule, c += a.class_row) {
            const int cls = *c;
            if (cls == 2) return there;
            if (cls == 0) continue;
            const bool any = words && (attn_word<kGradKV>(a, words, q) | attn_word<kGradKV>(a, words, q + 32));
            some |= __ballot_sync(0xffffffffu, any);
            if (some == there) return there;
        }
    }
    return some;
}

// The largest of a block's values.
__device__ __forceinline__ float attn_block_most(float most) {
    __shared__ float part[kDeltaThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
    __syncthreads();                   // the last call's are read
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kDeltaThreads / 32; ++i) most = fmaxf(most, part[i]);
    return most;
}

// fp16: the largest finite |v_j|^2 of the keys of part p of a batch entry's and key head's,
// of those that a query attends: what lies in masked places has no part in it.
template <typename T, int L>
__device__ __forceinline__ void attn_key_norms(const AttnArgs &a, int64_t slice, int p) {
    constexpr int V = 16 / sizeof(T), AT_ONCE = 4;
    const int d = threadIdx.x % L * V, b = (int)(slice / a.N), n = (int)(slice - (int64_t)b * a.N);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, groups = (a.S + 31) / 32;     // of 32 keys, one a warp
    const int begin = (int)((int64_t)groups * p / a.norms), end = (int)((int64_t)groups * (p + 1) / a.norms);
    float most = 0.0f;
    for (int t = begin + warp; t < end; t += kDeltaThreads / 32) {
        uint32_t some = 0u;
#pragma unroll
        for (int i0 = 0; i0 < L; i0 += AT_ONCE) {
            uint4 x[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int key = 32 * t + (i0 + i) * (32 / L) + lane / L;
                x[i] = key < a.S && d < a.D ? ldg16(attn_at<T>(a, a.v, b, key, n) + d) : make_uint4(0u, 0u, 0u, 0u);
            }
            if (i0 == 0) some = attn_attended(a, b, n, 32 * t);
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                float fx[V], square = 0.0f;
                unpack16<T>(fx, x[i]);
#pragma unroll
                for (int k = 0; k < V; ++k) square = fmaf(fx[k], fx[k], square);
#pragma unroll
                for (int off = L / 2; off > 0; off >>= 1) square += __shfl_xor_sync(0xffffffffu, square, off);
                const bool on = (some >> ((i0 + i) * (32 / L) + lane / L)) & 1u;
                if (on && isfinite(square)) most = fmaxf(most, square);
            }
        }
    }
    most = attn_block_most(most);
    if (threadIdx.x == 0) a.norm_v[slice * a.norms + p] = most;
}

// The queries' stat: the row sums delta = sum over channels of dO out, L lanes a row
// of 16 bytes each, beside the forward's lse. NORMS (fp16): rows by batch entry and key
// head, in a.norms parts each, and of each part the largest finite |dO_i|^2 of queries that
// attend a key; and the keys' norms, by other blocks.
template <typename T, int L, bool NORMS>
__global__ void __launch_bounds__(kDeltaThreads) attn_delta_kernel(const AttnArgs a) {
    constexpr int V = 16 / sizeof(T), per = kDeltaThreads / L, AT_ONCE = 4;
    attn_after();
    const int lane = threadIdx.x % L, d = lane * V, heads = NORMS ? a.G : a.M;
    const int64_t step = NORMS ? per : (int64_t)gridDim.x * per;
    const int64_t parts = NORMS ? (int64_t)a.B * a.N * a.norms : gridDim.x;
    for (int64_t t = blockIdx.x; t < (NORMS ? 2 * parts : parts); t += gridDim.x) {
        const int64_t slice = NORMS ? t % parts / a.norms : 0;         // b N + n
        const int p = NORMS ? (int)(t % parts - slice * a.norms) : 0;
        if (NORMS && t >= parts) {
            attn_key_norms<T, L>(a, slice, p);
            continue;
        }
        const int64_t all = NORMS ? (int64_t)a.stat_row * a.G : (int64_t)a.B * a.stat_row * a.M;
        const int64_t begin = NORMS ? all * p / a.norms : (int64_t)blockIdx.x * per, rows = NORMS ? all * (p + 1) / a.norms : all;
        float most_do = 0.0f;
        for (int64_t r0 = begin + threadIdx.x / L; r0 - threadIdx.x / L < rows; r0 += AT_ONCE * step) {
            uint4 x[AT_ONCE], y[AT_ONCE], z[AT_ONCE];
            float *to[AT_ONCE];
            float lse[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int64_t r = r0 + i * step, bq = r / heads;
                int m = (int)(r - bq * heads), b, q;
                if (NORMS) {
                    b = (int)(slice / a.N);
                    q = (int)bq;
                    m += (int)(slice - (int64_t)b * a.N) * a.G;
                } else {
                    b = (int)(bq / a.stat_row);
                    q = (int)(bq - (int64_t)b * a.stat_row);
                }
                to[i] = r < rows ? attn_stat(a, b, m, q) : nullptr;
                x[i] = y[i] = z[i] = make_uint4(0u, 0u, 0u, 0u);
                lse[i] = -INFINITY;
                if (r < rows && q < a.Q) {
                    if (NORMS || lane == 0) lse[i] = a.lse[((int64_t)b * a.M + m) * a.Q + q];
                    if (d < a.D) {     // these three lie alike
                        const T *go = attn_at<T>(a, a.go, b, q, m) + d;
                        const int64_t at = go - static_cast<const T *>(a.go.p);
                        x[i] = ldg16(go);
                        y[i] = ldg16(static_cast<const T *>(a.o.p) + at);
                        if (a.rest) z[i] = ldg16(static_cast<const T *>(a.rest) + at);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                float fx[V], fy[V], fz[V], dot = 0.0f, square = 0.0f;
                unpack16<T>(fx, x[i]);
                unpack16<T>(fy, y[i]);
                unpack16<T>(fz, z[i]);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    dot = fmaf(fx[k], fy[k] + fz[k], dot);
                    if (NORMS) square = fmaf(fx[k], fx[k], square);
                }
#pragma unroll
                for (int off = L / 2; off > 0; off >>= 1) {
                    dot += __shfl_xor_sync(0xffffffffu, dot, off);
                    if (NORMS) square += __shfl_xor_sync(0xffffffffu, square, off);
                }
                if (NORMS && isfinite(square) && lse[i] != -INFINITY) most_do = fmaxf(most_do, square);
                if (to[i] && lane == 0) {      // past the last query: -infinity and 0
                    to[i][0] = a.up - attn_lse2(lse[i]);
                    to[i][2] = -dot;
                }
            }
        }
        if (!NORMS) return;
        most_do = attn_block_most(most_do);
        if (threadIdx.x == 0) a.norm_do[t] = most_do;
    }
}

template <typename T> cudaError_t launch_delta(const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    constexpr bool NORMS = std::is_same<T, __half>::value;
    const int lanes = a.D * (int)sizeof(T) / 16;
    if (lanes <= 4) return launch_after(a.chained, attn_delta_kernel<T, 4, NORMS>, blocks, kDeltaThreads, 0, stream, a);
    if (lanes <= 8) return launch_after(a.chained, attn_delta_kernel<T, 8, NORMS>, blocks, kDeltaThreads, 0, stream, a);
    if (lanes <= 16) return launch_after(a.chained, attn_delta_kernel<T, 16, NORMS>, blocks, kDeltaThreads, 0, stream, a);
    return launch_after(a.chained, attn_delta_kernel<T, 32, NORMS>, blocks, kDeltaThreads, 0, stream, a);
}

// Sums of the splits: a warp a row, four channels a lane, and where that leaves lanes the
// splits in turn over groups of LD of them, so that all loads are under way together.
// Forward: each split's sums are relative to its own maximum, and its weight is exp2 of
// the distance. At most 64 splits.
template <typename T, int LD>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a, int mode) {
    constexpr int GROUPS = 32 / LD;
    attn_after();
    const int lane = threadIdx.x & 31, group = lane / LD, d = lane % LD * 4;
    const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32, step = a.part_rows * a.D;
    if (row >= a.part_rows) return;
    float weight[2] = {1.0f, 1.0f}, base = 0.0f, sum = 1.0f;       // of splits lane, lane + 32
    if (mode == kForward) {
        const float2 *ml = reinterpret_cast<const float2 *>(a.part + a.splits * step) + row;
        float2 mine[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            mine[i] = lane + 32 * i < a.splits ? ml[(lane + 32 * i) * a.part_rows] : make_float2(-INFINITY, 0.0f);
        float top = fmaxf(mine[0].x, mine[1].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        base = top == -INFINITY ? 0.0f : top;
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            weight[i] = exp2f(mine[i].x - base);
            sum = fmaf(weight[i], mine[i].y, sum);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
    for (int which = 0; which < (mode == kGradKV ? 2 : 1); ++which) {
        const float *from = a.part + which * a.splits * step + row * a.D + d;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int s0 = 0; s0 < a.splits; s0 += GROUPS) {
            const int s = s0 + group;
            const float lo = __shfl_sync(0xffffffffu, weight[0], s & 31), hi = __shfl_sync(0xffffffffu, weight[1], s & 31);
            if (s < a.splits && d < a.D) {
                const float4 v = *reinterpret_cast<const float4 *>(from + s * step);
                const float f = s < 32 ? lo : hi;
                acc = make_float4(fmaf(f, v.x, acc.x), fmaf(f, v.y, acc.y), fmaf(f, v.z, acc.z), fmaf(f, v.w, acc.w));
            }
        }
#pragma unroll
        for (int off = LD; off < 32; off <<= 1) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
        }
        if (group > 0 || d >= a.D) continue;
        const float f = mode == kForward ? (sum == 0.0f ? 0.0f : 1.0f / sum) : mode == kGradQ || which ? a.scale : 1.0f;
        void *to = mode == kForward ? a.out : mode == kGradQ ? a.gq : which ? a.gk : a.gv;
        const float v[4] = {acc.x * f, acc.y * f, acc.z * f, acc.w * f};
#pragma unroll
        for (int k = 0; k < 4; ++k) attn_put<T>(a, to, mode == kForward ? a.rest : nullptr, row * a.D + d + k, v[k]);
    }
    if (mode == kForward && a.lse && lane == 0) {
        const int m = (int)(row % a.M);
        const int64_t bq = row / a.M;
        attn_put_lse(a, (int)(bq / a.Q), m, (int)(bq % a.Q), sum == 0.0f ? -INFINITY : (base + log2f(sum)) * kLn2);
    }
}

template <typename T> cudaError_t launch_join(int mode, const AttnArgs &a, cudaStream_t stream) {
    const int64_t blocks = ((a.part_rows + 3) / 4);
    if (a.D <= 16) return launch_after(true, attn_join_kernel<T, 4>, blocks, 128, 0, stream, a, mode);
    if (a.D <= 32) return launch_after(true, attn_join_kernel<T, 8>, blocks, 128, 0, stream, a, mode);
    if (a.D <= 64) return launch_after(true, attn_join_kernel<T, 16>, blocks, 128, 0, stream, a, mode);
    return launch_after(true, attn_join_kernel<T, 32>, blocks, 128, 0, stream, a, mode);
}

}  // namespace

cudaError_t launch_attention_pack(const AttnMaskSource &m, uint32_t *by_query, int words_q, uint32_t *by_key,
                                  int words_k, uint8_t *classes, int granules, cudaStream_t stream) {
    const int64_t blocks = (int64_t)m.B * m.M * ((m.Q + kPackQ - 1) / kPackQ) * (granules / 2);
    return launch_after(false, attn_pack_kernel, blocks, 256, 0, stream, m, by_query, words_q, by_key, words_k, classes, granules);
}

cudaError_t launch_attention_delta(const AttnArgs &a, int64_t blocks, msda_dtype_t dt, cudaStream_t stream) {
    return dt == MSDA_F32 ? launch_delta<float>(a, blocks, stream)
         : dt == MSDA_BF16 ? launch_delta<__nv_bfloat16>(a, blocks, stream) : launch_delta<__half>(a, blocks, stream);
}

cudaError_t launch_attention_join(int mode, const AttnArgs &a, msda_dtype_t dt, cudaStream_t stream) {
    return dt == MSDA_F32 ? launch_join<float>(mode, a, stream)
         : dt == MSDA_BF16 ? launch_join<__nv_bfloat16>(mode, a, stream) : launch_join<__half>(mode, a, stream);
}

}  // namespace msda
