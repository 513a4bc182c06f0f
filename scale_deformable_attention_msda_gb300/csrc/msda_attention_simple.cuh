// Attention in fp32 arithmetic: tiles of 64 rows by 64 columns in shared memory,
// scores and products with fused multiply-adds, 4 x 4 scores a thread. All of it is
// fp32; no operand is rounded to fewer bits.
//
// What bounds it: the instructions around the multiply-adds (a shared-memory load of 16
// bytes for every 8 of them, exponentials, addresses) and their latencies: 1024 x 1024 of
// 16 heads, D 32 / 64 / 128: forward 93 / 149 / 345 us (23 to 29 TFLOP/s of 75), backward
// 291 / 469 / 1,070. 300 queries of 16 heads, D 32, where a block has one tile or two:
// 19 and 50 us. 8 x 4 scores and 128 threads, with packed multiply-adds: 114 us forward
// instead of 101, 617 instead of 467 at D 128. The next tile's loads under way during the
// arithmetic: no gain at D 32 (95.6 us, 96.4), slower at D 64 (509 us backward, 468). Three
// blocks of an SM at D 32: 47 us instead of 50 for the 300 queries' backward, but 342
// instead of 287 for 1024.
#pragma once

#include "msda_attention.cuh"
#include "msda_attention_host.h"

namespace msda {

constexpr int kSimpleTile = 64, kSimpleThreads = 256;

template <int DP> struct SimpleShared {
    static constexpr int kLd = DP + 4, kLdP = kSimpleTile + 4;
    float a1[kSimpleTile * kLd], a2[kSimpleTile * kLd], x1[kSimpleTile * kLd], x2[kSimpleTile * kLd];
    float p[kSimpleTile * kLdP], ds[kSimpleTile * kLdP];
    float lse2[kSimpleTile], delta[kSimpleTile];
    float stat[2][kSimpleTile];        // forward: a bad row's reference maximum and sum
    int bad[kSimpleTile];
};

// This thread's share of 64 rows of D channels on their way to shared memory; zeros where
// `row` gives NULL and past D.
template <int DP> struct SimpleRows {
    static constexpr int N = kSimpleTile * (DP / 4) / kSimpleThreads, STEP = kSimpleThreads / (DP / 4);
    float4 v[N];
    template <class F> __device__ __forceinline__ void fetch(int D, F row) {
        const int r = threadIdx.x / (DP / 4), d = threadIdx.x % (DP / 4) * 4;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float *from = row(r + i * STEP);
            v[i] = from && d < D ? __ldg(reinterpret_cast<const float4 *>(from + d)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    }
    __device__ __forceinline__ void put(float *to) const {
        const int r = threadIdx.x / (DP / 4), d = threadIdx.x % (DP / 4) * 4;
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<float4 *>(to + (r + i * STEP) * (DP + 4) + d) = v[i];
    }
};

// s[i][j] = row 4 ty + i of a times row tx + 16 j of x.
template <int DP>
__device__ __forceinline__ void simple_dot(float (&s)[4][4], const float *a, const float *x, int ty, int tx) {
    constexpr int ld = DP + 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 u[4], v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const float4 *>(a + (4 * ty + i) * ld + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float4 *>(x + (tx + 16 * j) * ld + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i][j] = fmaf(u[i].x, v[j].x, fmaf(u[i].y, v[j].y, fmaf(u[i].z, v[j].z, fmaf(u[i].w, v[j].w, s[i][j]))));
    }
}

// acc[i][k] += sum over 64 columns of p[4 ty + i][c] * x[c][channel(k)]; thread tx has
// the DP / 16 channels tx (DP / 16) + k.
template <int DP>
__device__ __forceinline__ void simple_product(float (&acc)[4][DP / 16], const float *p, const float *x, int ty, int tx) {
    constexpr int ld = DP + 4, E = DP / 16;
#pragma unroll 2
    for (int c = 0; c < kSimpleTile; c += 4) {
        float4 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const float4 *>(p + (4 * ty + i) * (kSimpleTile + 4) + c);
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
            float v[E];
#pragma unroll
            for (int k = 0; k < E; k += 2)
                *reinterpret_cast<float2 *>(v + k) = *reinterpret_cast<const float2 *>(x + (c + cc) * ld + tx * E + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = cc == 0 ? u[i].x : cc == 1 ? u[i].y : cc == 2 ? u[i].z : u[i].w;
#pragma unroll
                for (int k = 0; k < E; ++k) acc[i][k] = fmaf(w, v[k], acc[i][k]);
            }
        }
    }
}

// E channels of a row from d on, two at a time (E divides 8, and D is a multiple of 8).
// The sums are of the output's type: its rounding leaves nothing.
template <int MODE, int E>
__device__ __forceinline__ void simple_store(const AttnArgs &a, const AttnRows &w, int r, int split, int which, int d, const float (&v)[E], float f) {
    const int len = MODE == kGradKV ? a.S : a.Q, heads = MODE == kGradKV ? a.N : a.M;
    const int64_t row = ((int64_t)w.b * len + w.row_pos(r)) * heads + w.row_head(r);
    if (!attn_ok(a, row, a.part_rows)) return;
    const bool parts = a.splits > 1;
    float *to = parts ? a.part + ((int64_t)(which * a.splits + split) * a.part_rows + row) * a.D
                      : static_cast<float *>(MODE == kForward ? a.out : MODE == kGradQ ? a.gq : which ? a.gk : a.gv) + row * a.D;
    if (parts) f = 1.0f;
#pragma unroll
    for (int k = 0; k < E; k += 2) {
        *reinterpret_cast<float2 *>(to + d + k) = make_float2(v[k] * f, v[k + 1] * f);
        if (MODE == kForward && !parts && a.rest) *reinterpret_cast<float2 *>(static_cast<float *>(a.rest) + row * a.D + d + k) = make_float2(0.0f, 0.0f);
    }
}

template <int MODE, int DP>
__global__ void __launch_bounds__(kSimpleThreads, simple_blocks(DP)) attn_simple_kernel(const AttnArgs a) {
    constexpr int R = kSimpleTile, C = kSimpleTile, E = DP / 16, LDP = SimpleShared<DP>::kLdP;
    extern __shared__ __align__(16) unsigned char raw[];
    SimpleShared<DP> &sh = *reinterpret_cast<SimpleShared<DP> *>(raw);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, lane = threadIdx.x & 31;
    const int split = blockIdx.x % a.splits;
    const AttnRows w = attn_rows<MODE, R>(a, blockIdx.x / a.splits);
    const int64_t tiles = attn_column_tiles<MODE, C>(a);
    const int64_t j0 = tiles * split / a.splits, j1 = tiles * (split + 1) / a.splits;
    attn_after();

    auto row_of = [&](const AttnTensor &t) {
        return [&, t](int r) { return w.valid(r) ? attn_at<float>(a, t, w.b, w.row_pos(r), w.row_head(r)) : nullptr; };
    };
    SimpleRows<DP> x1, x2;
    x1.fetch(a.D, row_of(MODE == kGradKV ? a.k : a.q));
    if (MODE != kForward) x2.fetch(a.D, row_of(MODE == kGradKV ? a.v : a.go));
    x1.put(sh.a1);
    if (MODE != kForward) x2.put(sh.a2);
    if (threadIdx.x < R) sh.bad[threadIdx.x] = 0;

    float acc1[4][E], acc2[4][E], top[4], sum[4], lse2[4], delta[4];
    const uint32_t *words[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        top[i] = -INFINITY;
        sum[i] = delta[i] = 0.0f;
        lse2[i] = INFINITY;
        words[i] = nullptr;
        if (MODE != kGradKV && w.valid(r)) {
            words[i] = attn_word_row<MODE>(a, w.b, w.row_head(r), w.row_pos(r));
            if (MODE == kGradQ) {
                const float *st = attn_stat(a, w.b, w.row_head(r), w.row_pos(r));
                lse2[i] = -st[0];
                delta[i] = -st[2];
            }
        }
#pragma unroll
        for (int k = 0; k < E; ++k) acc1[i][k] = acc2[i][k] = 0.0f;
    }

    const int len = MODE == kGradKV ? a.Q : a.S;
    for (int64_t j = j0; j < j1; ++j) {
        int pos, head;
        attn_columns<MODE, C>(a, w, j, &pos, &head);
        const int cls = attn_class<MODE, C>(a, w, pos, head);
        if (!cls) continue;
        auto column_of = [&](const AttnTensor &t) {
            return [&, t](int c) { return pos + c < len ? attn_at<float>(a, t, w.b, pos + c, head) : nullptr; };
        };
        x1.fetch(a.D, column_of(MODE == kGradKV ? a.q : a.k));
        x2.fetch(a.D, column_of(MODE == kGradKV ? a.go : a.v));
        __syncthreads();
        x1.put(sh.x1);
        x2.put(sh.x2);
        if (MODE == kGradKV) {
            if (threadIdx.x < C) {
                const float *st = attn_stat(a, w.b, head, pos + threadIdx.x);
                sh.lse2[threadIdx.x] = -st[0];
                sh.delta[threadIdx.x] = -st[2];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (w.valid(4 * ty + i)) words[i] = attn_word_row<MODE>(a, w.b, head, w.row_pos(4 * ty + i));
        }
        __syncthreads();

        float s[4][4], dp[4][4];
        simple_dot<DP>(s, sh.a1, sh.x1, ty, tx);
        if (MODE != kForward) simple_dot<DP>(dp, sh.a2, sh.x2, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bool on[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = tx + 16 * k;
                on[k] = cls == 2 || ((attn_word<MODE>(a, words[i], pos + (c & ~31)) >> (c & 31)) & 1u);
            }
            float *prow = sh.p + (4 * ty + i) * LDP, *drow = sh.ds + (4 * ty + i) * LDP;
            if (MODE == kForward) {
                float m = top[i];
#pragma unroll
                for (int k = 0; k < 4; ++k) m = fmaxf(m, on[k] ? s[i][k] : -INFINITY);
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                const float base = m == -INFINITY ? 0.0f : m, old = top[i] == -INFINITY ? 0.0f : exp2f((top[i] - base) * a.c);
                top[i] = m;
                sum[i] *= old;
#pragma unroll
                for (int k = 0; k < E; ++k) acc1[i][k] *= old;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float p = on[k] ? exp2f((s[i][k] - base) * a.c) : 0.0f;
                    sum[i] += p;
                    prow[tx + 16 * k] = p;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = tx + 16 * k;
                    const float l = MODE == kGradKV ? sh.lse2[c] : lse2[i], e = MODE == kGradKV ? sh.delta[c] : delta[i];
                    const bool use = on[k] && l != INFINITY;
                    const float p = use ? exp2f(fmaf(s[i][k], a.c, -l)) : 0.0f;
                    if (MODE == kGradKV) prow[c] = p;
                    drow[c] = use ? p * (dp[i][k] - e) : 0.0f;
                }
            }
        }
        __syncthreads();
        if (MODE != kGradQ) simple_product<DP>(acc1, sh.p, sh.x2, ty, tx);
        if (MODE != kForward) simple_product<DP>(acc2, sh.ds, sh.x1, ty, tx);
    }

#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (MODE == kForward) {
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
        }
        bool finite = true;
#pragma unroll
        for (int k = 0; k < E; ++k) finite = finite && isfinite(acc1[i][k]) && isfinite(acc2[i][k]);
        const uint32_t vote = __ballot_sync(0xffffffffu, !finite) & (lane < 16 ? 0xffffu : 0xffff0000u);
        if (!w.valid(r)) continue;
        const float m2 = top[i] == -INFINITY ? 0.0f : top[i] * a.c;
        if (MODE == kForward && tx == 0) {
            const int64_t row = ((int64_t)w.b * a.Q + w.row_pos(r)) * a.M + w.row_head(r);
            if (a.splits > 1) {
                float *ml = a.part + (int64_t)a.splits * a.part_rows * a.D + 2 * ((int64_t)split * a.part_rows + row);
                ml[0] = sum[i] == 0.0f ? -INFINITY : m2;
                ml[1] = sum[i];
            } else if (a.lse) {
                attn_put_lse(a, w.b, w.row_head(r), w.row_pos(r), sum[i] == 0.0f ? -INFINITY : (m2 + log2f(sum[i])) * kLn2);
            }
        }
        if (vote && a.classes) {       // not finite, and the mask may be why
            if (tx == 0) {
                sh.bad[r] = 1;
                sh.stat[0][r] = m2;
                sh.stat[1][r] = sum[i];
            }
        }
        const float f = MODE == kForward ? (sum[i] == 0.0f ? 0.0f : 1.0f / sum[i]) : a.scale;
        if (tx * E >= a.D) continue;
        if (MODE != kGradQ) simple_store<MODE, E>(a, w, r, split, 0, tx * E, acc1[i], MODE == kForward ? f : 1.0f);
        if (MODE != kForward) simple_store<MODE, E>(a, w, r, split, MODE == kGradKV, tx * E, acc2[i], f);
    }
    __syncthreads();
    // a warp has every eighth row
    constexpr int WARPS = kSimpleThreads / 32;
    const int mine = threadIdx.x / 32 + WARPS * lane;
    const bool bad = lane < R / WARPS && sh.bad[mine];
    uint32_t again = __ballot_sync(0xffffffffu, bad);
    if (again) again = __ballot_sync(0xffffffffu, attn_spoiled<float, MODE, C>(a, w, bad ? mine : -1, j0, j1, MODE == kForward && bad && !isfinite(sh.stat[1][mine])));
    for (; again; again &= again - 1) {
        const int r = threadIdx.x / 32 + WARPS * (__ffs(again) - 1);
        float e1[4], e2[4];
        attn_exact_row<float, MODE, C>(a, w, r, j0, j1, MODE == kForward ? sh.stat[0][r] : 0.0f, e1, e2);
        const float f = MODE != kForward ? a.scale : sh.stat[1][r] == 0.0f ? 0.0f : 1.0f / sh.stat[1][r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = lane + 32 * i;
            if (d >= a.D) continue;
            if (MODE != kGradQ) attn_store<float, MODE>(a, w, r, split, 0, d, e1[i], MODE == kForward ? f : 1.0f);
            if (MODE != kForward) attn_store<float, MODE>(a, w, r, split, MODE == kGradKV, d, e2[i], f);
        }
    }
}

template <int MODE, int DP>
cudaError_t launch_simple_d(const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    constexpr int bytes = (int)sizeof(SimpleShared<DP>);
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(attn_simple_kernel<MODE, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    return launch_after(a.chained, attn_simple_kernel<MODE, DP>, blocks, kSimpleThreads, bytes, stream, a);
}
template <int MODE>
cudaError_t launch_simple_mode(const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    return a.D <= 32 ? launch_simple_d<MODE, 32>(a, blocks, stream)
         : a.D <= 64 ? launch_simple_d<MODE, 64>(a, blocks, stream)
                     : launch_simple_d<MODE, 128>(a, blocks, stream);
}
inline cudaError_t launch_simple(int mode, const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    return mode == kForward ? launch_simple_mode<kForward>(a, blocks, stream)
         : mode == kGradQ   ? launch_simple_mode<kGradQ>(a, blocks, stream)
                            : launch_simple_mode<kGradKV>(a, blocks, stream);
}

}  // namespace msda
