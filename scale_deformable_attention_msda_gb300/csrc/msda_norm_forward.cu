// Layer norm, forward: out = (s - mean) * rstd * weight + bias over the C
// channels of each row of s = x + residual, mean and biased variance per row.
//
// A row is read once and stays in registers: its mean, then the sum of squared
// distances from that mean (no difference of large sums), then the output. All
// arithmetic in fp32; s is not rounded before it is normalised.
#include "msda_norm.cuh"

namespace msda {

template <typename T, typename W, int G, int KV, int VEC>
__global__ void __launch_bounds__(G > 0 ? 256 : (VEC == 1 ? 1024 : 512))
norm_forward_kernel(const NormArgs a) {
    __shared__ BlockScratch<1> scratch;
    int turn = 0;
    const int threads = G == 0 ? blockDim.x : G;
    const int t = G == 0 ? threadIdx.x : threadIdx.x % G;
    const int64_t first = G == 0 ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
    const int64_t step = G == 0 ? gridDim.x : (int64_t)gridDim.x * (blockDim.x / G);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const W *w = static_cast<const W *>(a.weight), *b = static_cast<const W *>(a.bias);
    const int C = a.C;
    const int64_t extent = a.N * C;
    const float inv_C = 1.0f / (float)C;
    // rows are walked by whole warps: a lane of a group past the last row works on zeros
    const int64_t warp_first = G == 0 ? first : (int64_t)blockIdx.x * (blockDim.x / G) + (threadIdx.x & ~31) / (G == 0 ? 1 : G);
    for (int64_t row = first, lead = warp_first; lead < a.N; row += step, lead += step) {
        const bool valid = row < a.N;
        const int64_t base = row * C;
        float s[KV][VEC];
        bool mine[KV];
        float sum[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const int c = (k * threads + t) * VEC;
            mine[k] = valid && c < C && span_ok(a.err, base + c, VEC, extent);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[k][i] = 0.0f;
            if (mine[k]) {
                Raw<T, VEC> r;
                r.load(x + base + c);
                r.unpack(s[k]);
            }
        }
        if (res) {
#pragma unroll
            for (int k = 0; k < KV; ++k) {
                const int c = (k * threads + t) * VEC;
                if (mine[k]) {
                    Raw<T, VEC> r;
                    float e[VEC];
                    r.load(res + base + c);
                    r.unpack(e);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s[k][i] += e[i];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < KV; ++k) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[0] += s[k][i];
        }
        row_sum<G>(sum, &scratch, turn);
        const float mean = sum[0] * inv_C;
        float sq[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < KV; ++k) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = mine[k] ? s[k][i] - mean : 0.0f;
                sq[0] = fmaf(d, d, sq[0]);
            }
        }
        row_sum<G>(sq, &scratch, turn);
        const float rstd = 1.0f / sqrtf(sq[0] * inv_C + (float)a.eps);
        if (t == 0 && valid && a.mean && span_ok(a.err, row, 1, a.N)) {
            static_cast<float *>(a.mean)[row] = mean;
            static_cast<float *>(a.rstd)[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const int c = (k * threads + t) * VEC;
            if (!mine[k]) continue;
            if (a.sum) Raw<T, VEC>::store(static_cast<T *>(a.sum) + base + c, s[k]);
            float g[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) g[i] = (s[k][i] - mean) * rstd;
            if (w) {
                Raw<W, VEC> r;
                float e[VEC];
                r.load(w + c);
                r.unpack(e);
#pragma unroll
                for (int i = 0; i < VEC; ++i) g[i] *= e[i];
            }
            if (b) {
                Raw<W, VEC> r;
                float e[VEC];
                r.load(b + c);
                r.unpack(e);
#pragma unroll
                for (int i = 0; i < VEC; ++i) g[i] += e[i];
            }
            Raw<T, VEC>::store(static_cast<T *>(a.out) + base + c, g);
        }
    }
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

// Rows of any length, one block each, read three times (the later reads hit
// the caches): fp64, and rows too long for the registers.
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

template <typename T, typename W>
static cudaError_t launch_forward_t(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
#define FWD(g, kv, vec)                                                                            \
    if (p.G == g && p.KV == kv) {                                                                  \
        norm_forward_kernel<T, W, g, kv, vec><<<p.blocks, p.threads, 0, stream>>>(a);              \
        return cudaGetLastError();                                                                 \
    }
    if (p.general) {
        norm_forward_general_kernel<T, W><<<p.blocks, p.threads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    if (p.vec) {
        constexpr int V = Vec16<T>::N;
        FWD(4, 1, V) FWD(8, 1, V) FWD(16, 1, V) FWD(32, 1, V) FWD(32, 2, V)
        FWD(0, 1, V) FWD(0, 2, V) FWD(0, 4, V)
    } else {
        FWD(32, 1, 1) FWD(32, 4, 1) FWD(32, 8, 1) FWD(0, 4, 1) FWD(0, 8, 1)
    }
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
