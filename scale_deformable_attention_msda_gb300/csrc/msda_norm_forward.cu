// Layer norm, forward: out = (s - mean) * rstd * weight + bias over the C
// channels of each row of s = x + residual, mean and biased variance per row.
//
// A row is read once and stays in registers: its mean, then the sum of squared
// distances from that mean (no difference of large sums), then the output. All
// arithmetic in fp32; s is not rounded before it is normalised.
#include "msda_norm.cuh"

namespace msda {

// S: rows whose copies are under way while one is worked on. A thread copies
// what it reads itself, so its own wait is all the order the copies need.
template <typename T, typename W, int G, int KV, bool RAGGED, int S, int TH>
__global__ void __launch_bounds__(TH) norm_forward_kernel(const NormArgs a) {
    constexpr int V = Vec16<T>::N, P = V / 2;
    __shared__ BlockScratch<1> scratch;
    extern __shared__ uint4 ring[];      // (S, tensors, KV, threads)
    int turn = 0;
    const int C = a.C;
    const RowMap<G, KV, V, RAGGED, TH> map(a);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const W *w = static_cast<const W *>(a.weight), *b = static_cast<const W *>(a.bias);
    const int64_t extent = a.N * C, hop = map.step * C;
    const float inv_C = 1.0f / (float)C;
    const int plane = G == 0 ? blockDim.x : TH;   // a thread's slots are this far apart
    const int tensors = res ? 2 : 1, tall = tensors * KV * plane;
    int64_t here = map.start(C), ahead = here;
    int64_t coming = map.first;          // the row at `ahead`
    auto fetch = [&](uint4 *to) {
        const bool there = coming < a.N;
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            map.fetch(to + k * plane, x, ahead, k, there, extent, a.err);
            if (res) map.fetch(to + (KV + k) * plane, res, ahead, k, there, extent, a.err);
        }
        coming += map.step;
        ahead += hop;
        fetch_commit();
    };
    uint4 *const begin = ring + threadIdx.x, *slot = begin;
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(begin + i * tall);
    float2 pw[KV][P], pb[KV][P];
#pragma unroll
    for (int k = 0; k < KV; ++k) {
        const int c = map.channel(k);
        if (RAGGED) {
            load_params_masked<W, V>(pw[k], w, c, C, 1.0f);
            load_params_masked<W, V>(pb[k], b, c, C, 0.0f);
        } else {
            load_params<W, V>(pw[k], map.held(k) ? w : nullptr, c, 1.0f);
            load_params<W, V>(pb[k], map.held(k) ? b : nullptr, c, 0.0f);
        }
    }
    for (int64_t row = map.first, lead = map.lead; lead < a.N; row += map.step, lead += map.step, here += hop) {
        const bool valid = G == 0 || G == 32 || row < a.N;
        float2 s[KV][P];
        float2 acc = both(0.0f);
        fetch_wait<S - 1>();
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            unpack_pairs<T>(s[k], slot[k * plane]);
            if (res) {
                float2 e[P];
                unpack_pairs<T>(e, slot[(KV + k) * plane]);
#pragma unroll
                for (int i = 0; i < P; ++i) s[k][i] = add2(s[k][i], e[i]);
            }
            if (a.sum && valid && map.held(k)) map.store(static_cast<T *>(a.sum), here, k, C, s[k]);
            if (RAGGED && !map.whole(k, C)) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if (!map.has(k, 2 * i, C)) s[k][i].x = 0.0f;
                    if (!map.has(k, 2 * i + 1, C)) s[k][i].y = 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) acc = add2(acc, s[k][i]);
        }
        float v[1] = {acc.x + acc.y};
        row_sum<G>(v, &scratch, turn, map.threads, map.index);
        fetch(slot);
        slot = slot + tall == begin + S * tall ? begin : slot + tall;
        const float mean = v[0] * inv_C;
        acc = both(0.0f);
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const float m = map.held(k) ? -mean : 0.0f;      // a slot without a granule stays zero
#pragma unroll
            for (int i = 0; i < P; ++i) s[k][i] = add2(s[k][i], both(m));
            if (RAGGED && !map.whole(k, C)) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if (!map.has(k, 2 * i, C)) s[k][i].x = 0.0f;
                    if (!map.has(k, 2 * i + 1, C)) s[k][i].y = 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) acc = fma2(s[k][i], s[k][i], acc);
        }
        v[0] = acc.x + acc.y;
        row_sum<G>(v, &scratch, turn, map.threads, map.index);
        const float rstd = rsqrtf(fmaf(v[0], inv_C, (float)a.eps));     // within 2 ulp
        if (map.t == 0 && valid && a.mean && span_ok(a.err, row, 1, a.N)) {
            static_cast<float *>(a.mean)[row] = mean;
            static_cast<float *>(a.rstd)[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < KV; ++k) {
#pragma unroll
            for (int i = 0; i < P; ++i) s[k][i] = fma2(mul2(s[k][i], both(rstd)), pw[k][i], pb[k][i]);
            if (valid && map.held(k)) map.store(static_cast<T *>(a.out), here, k, C, s[k]);
        }
    }
    fetch_wait<0>();
}

// Accumulation type of the general kernels: fp32 for 16- and 32-bit data.
template <typename T> struct Acc { using type = float; };
template <> struct Acc<double> { using type = double; };
template <typename T> __device__ __forceinline__ typename Acc<T>::type to_acc(T v) { return Elem<T>::to_f(v); }
template <> __device__ __forceinline__ double to_acc<double>(double v) { return v; }
template <typename T, typename A> __device__ __forceinline__ T from_acc(A v) { return Elem<T>::from_f(v); }
template <> __device__ __forceinline__ double from_acc<double, double>(double v) { return v; }

// Sum over a block, in every thread.
template <typename A> __device__ __forceinline__ A block_sum(A v, A *scratch) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += scratch[i];
    return v;
}

// Rows of any length and alignment, one block each, read three times (the
// later reads hit the caches): fp64, rows too long for the registers, pointers
// off a 16-byte boundary.
template <typename T, typename W>
__global__ void __launch_bounds__(512) norm_forward_general_kernel(const NormArgs a) {
    using A = typename Acc<T>::type;
    __shared__ A scratch[kMaxWarps];
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const W *w = static_cast<const W *>(a.weight), *b = static_cast<const W *>(a.bias);
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const int64_t base = row * a.C;
        if (!span_ok(a.err, base, a.C, a.N * a.C)) continue;
        A v = 0;
        for (int c = threadIdx.x; c < a.C; c += blockDim.x)
            v += to_acc<T>(x[base + c]) + (res ? to_acc<T>(res[base + c]) : (A)0);
        const A mean = block_sum<A>(v, scratch) / (A)a.C;
        v = 0;
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            const A d = to_acc<T>(x[base + c]) + (res ? to_acc<T>(res[base + c]) : (A)0) - mean;
            v += d * d;
        }
        const A rstd = (A)1 / sqrt(block_sum<A>(v, scratch) / (A)a.C + (A)a.eps);
        if (threadIdx.x == 0 && a.mean) {
            static_cast<A *>(a.mean)[row] = mean;
            static_cast<A *>(a.rstd)[row] = rstd;
        }
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            const A s = to_acc<T>(x[base + c]) + (res ? to_acc<T>(res[base + c]) : (A)0);
            if (a.sum) static_cast<T *>(a.sum)[base + c] = from_acc<T, A>(s);
            A g = (s - mean) * rstd;
            if (w) g *= (A)to_acc<W>(w[c]);
            if (b) g += (A)to_acc<W>(b[c]);
            static_cast<T *>(a.out)[base + c] = from_acc<T, A>(g);
        }
    }
}

template <typename T, typename W, int G, int KV, bool RAGGED, int S, int TH>
static cudaError_t launch_rows(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    auto kernel = norm_forward_kernel<T, W, G, KV, RAGGED, S, TH>;
    const size_t smem = (size_t)S * (a.residual ? 2 : 1) * KV * p.threads * 16;
    if (smem > kDefaultShared) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.blocks, p.threads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, typename W>
static cudaError_t launch_forward_t(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
#define FWD(g, kv, r, s) \
    if (p.G == g && p.KV == kv && p.ragged == r) return launch_rows<T, W, g, kv, r, s, g == 0 ? 512 : kForwardThreads>(a, p, stream);
    if (p.general) {
        norm_forward_general_kernel<T, W><<<p.blocks, p.threads, 0, stream>>>(a);
        return cudaGetLastError();
    }
#ifdef NORM_TUNE
    NORM_TUNE
#else
    FWD(2, 2, false, 2) FWD(4, 2, false, 2) FWD(8, 2, false, 2) FWD(16, 2, false, 2) FWD(32, 2, false, 2)
    FWD(0, 2, false, 2) FWD(0, 4, false, 1)
    FWD(2, 2, true, 2) FWD(4, 2, true, 2) FWD(8, 2, true, 2) FWD(16, 2, true, 2) FWD(32, 2, true, 2)
    FWD(0, 2, true, 2) FWD(0, 4, true, 1)
#endif
#undef FWD
    return cudaErrorInvalidValue;
}

cudaError_t launch_norm_forward(const NormArgs &a, const NormPlan &p, msda_dtype_t dt,
                                msda_dtype_t pdt, cudaStream_t stream) {
    const bool wide = pdt == MSDA_F32;
    switch (dt) {
        case MSDA_F32: return launch_forward_t<float, float>(a, p, stream);
        case MSDA_BF16: return wide ? launch_forward_t<__nv_bfloat16, float>(a, p, stream)
                                    : launch_forward_t<__nv_bfloat16, __nv_bfloat16>(a, p, stream);
        case MSDA_F16: return wide ? launch_forward_t<__half, float>(a, p, stream)
                                   : launch_forward_t<__half, __half>(a, p, stream);
        case MSDA_F64:
            norm_forward_general_kernel<double, double><<<p.blocks, p.threads, 0, stream>>>(a);
            return cudaGetLastError();
    }
    return cudaErrorInvalidValue;
}

}  // namespace msda
