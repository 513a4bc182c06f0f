// Attention's forward in fp32 for at most four rows a key head: a token that is decoded, a
// class token, their query heads that share the key head.
//
// What bounds it: the keys and values, each read once. One query of 8 heads over 4 x 8,192
// keys of 64 channels, 134 MB: 25.3 us, 5.3 TB/s; the tiles of 64 rows 180. (16-bit data
// stays on the tensor cores, although their blocks have 128 rows to fill: one query of 16
// heads over 4 x 16,384 keys of 4 heads and 64 channels, fp16, takes 20.7 us there and 33
// in this form, which is bound by its exchanges and conversions.)
//
// L lanes hold a key's channels, 8 each, and a warp reads 32 / L keys and values at a
// time, U times that under way. Each lane has the queries' 8 channels, scaled, and 8
// channels of each row's sum in registers; a score is 8 products and log2(L) exchanges.
// Each group of L lanes keeps a maximum and a sum of its own, joined at the end: in the
// warp, in the block, and over the blocks that share the keys by attn_join_kernel.
// What lies in masked places is replaced by zeros.
#include "msda_attention_host.h"

namespace msda {
namespace {

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
struct Channels {                      // 8 of a row
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void get(float *v) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

template <int L, int R>
__global__ void __launch_bounds__(kFewThreads, 2) attn_few_kernel(const AttnArgs a, int64_t keys_a_split) {
    constexpr int KEYS = 32 / L, U = R == 4 ? 2 : 4, DP = 8 * L;
    __shared__ float part_acc[kFewWarps][R][DP], part_top[kFewWarps][R], part_sum[kFewWarps][R];
    attn_after();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, group = lane / L, d = lane % L * 8;
    const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
    AttnRows w;
    w.b = tile / a.N;
    w.pack = a.G;
    w.head = tile % a.N * a.G;
    w.pos = 0;
    w.count = a.Q;
    const int n = tile % a.N;
    const int64_t k0 = split * keys_a_split;
    const int k1 = (int)(k0 + keys_a_split < a.S ? k0 + keys_a_split : a.S);
    const bool mine = d < a.D;

    float q[R][8], acc[R][8], top[R], sum[R];
    const uint32_t *words[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        Channels x;
        x.zero();
        if (w.valid(r) && mine) x.load(attn_at<float>(a, a.q, w.b, w.row_pos(r), w.row_head(r)) + d);
        x.get(q[r]);
        words[r] = w.valid(r) ? attn_word_row<kForward>(a, w.b, w.row_head(r), w.row_pos(r)) : nullptr;
        top[r] = -INFINITY;
        sum[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[r][i] *= a.c;
            acc[r][i] = 0.0f;
        }
    }
    for (int64_t from = k0 + warp * (KEYS * U); from < k1; from += kFewWarps * KEYS * U) {
        Channels k[U], v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = (int)from + u * KEYS + group;
            k[u].zero();
            v[u].zero();
            if (key < k1 && mine) {
                k[u].load(attn_at<float>(a, a.k, w.b, key, n) + d);
                v[u].load(attn_at<float>(a, a.v, w.b, key, n) + d);
            }
        }
        uint32_t on = 0u;              // bit r U + u
        float s[R][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = (int)from + u * KEYS + group;
            float x[8];
            k[u].get(x);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float t = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) t = fmaf(q[r][i], x[i], t);
#pragma unroll
                for (int off = 1; off < L; off <<= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
                if (key < k1 && (!words[r] || ((attn_word<kForward>(a, words[r], key & ~31) >> (key & 31)) & 1u))) on |= 1u << (r * U + u);
                s[r][u] = (on >> (r * U + u)) & 1u ? t : -INFINITY;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float high = top[r];
#pragma unroll
            for (int u = 0; u < U; ++u) high = fmaxf(high, s[r][u]);
            const float base = high == -INFINITY ? 0.0f : high, f = exp2f(top[r] - base);
            top[r] = high;
            sum[r] *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[r][i] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[r][u] = exp2f(s[r][u] - base);
                sum[r] += s[r][u];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[8];
            v[u].get(x);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!((on >> (r * U + u)) & 1u)) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[r][i] = fmaf(s[r][u], x[i], acc[r][i]);
            }
        }
    }
    // a warp's groups, then the block's warps
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float high = top[r];
#pragma unroll
        for (int off = L; off < 32; off <<= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, off));
        const float f = exp2f(top[r] - (high == -INFINITY ? 0.0f : high));
        sum[r] *= f;
#pragma unroll
        for (int off = L; off < 32; off <<= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], off);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            acc[r][i] *= f;
#pragma unroll
            for (int off = L; off < 32; off <<= 1) acc[r][i] += __shfl_xor_sync(0xffffffffu, acc[r][i], off);
            if (group == 0) part_acc[warp][r][d + i] = acc[r][i];
        }
        if (lane == 0) {
            part_top[warp][r] = high;
            part_sum[warp][r] = sum[r];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < R * DP; i += kFewThreads) {
        const int r = i / DP, at = i % DP;
        if (!w.valid(r) || at >= a.D) continue;
        float high = -INFINITY, all = 0.0f, value = 0.0f;
#pragma unroll
        for (int j = 0; j < kFewWarps; ++j) high = fmaxf(high, part_top[j][r]);
        const float base = high == -INFINITY ? 0.0f : high;
#pragma unroll
        for (int j = 0; j < kFewWarps; ++j) {
            const float f = exp2f(part_top[j][r] - base);
            all = fmaf(f, part_sum[j][r], all);
            value = fmaf(f, part_acc[j][r][at], value);
        }
        if (at == 0) {
            const int64_t row = ((int64_t)w.b * a.Q + w.row_pos(r)) * a.M + w.row_head(r);
            if (a.splits > 1) {
                float *ml = a.part + (int64_t)a.splits * a.part_rows * a.D + 2 * ((int64_t)split * a.part_rows + row);
                ml[0] = all == 0.0f ? -INFINITY : base;
                ml[1] = all;
            } else if (a.lse) {
                attn_put_lse(a, w.b, w.row_head(r), w.row_pos(r), all == 0.0f ? -INFINITY : (base + log2f(all)) * kLn2);
            }
        }
        attn_store<float, kForward>(a, w, r, split, 0, at, value, all == 0.0f ? 0.0f : 1.0f / all);
    }
}

template <int L> cudaError_t launch_few(const AttnArgs &a, int64_t blocks, int64_t keys_a_split, cudaStream_t stream) {
    const int rows = a.Q * a.G;
    if (rows == 1) return launch_after(a.chained, attn_few_kernel<L, 1>, blocks, kFewThreads, 0, stream, a, keys_a_split);
    if (rows == 2) return launch_after(a.chained, attn_few_kernel<L, 2>, blocks, kFewThreads, 0, stream, a, keys_a_split);
    return launch_after(a.chained, attn_few_kernel<L, 4>, blocks, kFewThreads, 0, stream, a, keys_a_split);
}

}  // namespace

cudaError_t launch_attention_few(const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    const int64_t keys_a_split = (((int64_t)a.S + a.splits - 1) / a.splits + 31) / 32 * 32;
    return a.D <= 32 ? launch_few<4>(a, blocks, keys_a_split, stream)
         : a.D <= 64 ? launch_few<8>(a, blocks, keys_a_split, stream) : launch_few<16>(a, blocks, keys_a_split, stream);
}

}  // namespace msda
