// Layer norm, backward. With xh = (s - mean) * rstd and g = grad_out * weight,
//
//   grad_x      = rstd * (g - mean_c(g) - xh * mean_c(g * xh)) + grad_sum
//   grad_weight = sum over the rows of grad_out * xh
//   grad_bias   = sum over the rows of grad_out
//
// One pass: while a row is in registers its threads add its part of the column
// sums to fp32 registers of their own (a thread keeps the same channels for
// all its rows), and a block leaves one row of partial sums for a second
// kernel to add up in a fixed order. No atomics: results do not vary.
#include "msda_norm.cuh"

namespace msda {

template <typename T, typename W, int G, int KV, int VEC>
__global__ void __launch_bounds__(G > 0 ? 256 : (VEC == 1 ? 1024 : 512))
norm_backward_kernel(const NormArgs a) {
    __shared__ BlockScratch<2> scratch;
    extern __shared__ float columns[];   // G > 0: (groups of the block, 2, C)
    int turn = 0;
    const int threads = G == 0 ? blockDim.x : G;
    const int t = G == 0 ? threadIdx.x : threadIdx.x % G;
    const int64_t first = G == 0 ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
    const int64_t step = G == 0 ? gridDim.x : (int64_t)gridDim.x * (blockDim.x / G);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const T *dy = static_cast<const T *>(a.grad_out), *ds = static_cast<const T *>(a.grad_sum);
    const W *w = static_cast<const W *>(a.weight);
    T *dx = static_cast<T *>(a.grad_x);
    const float *mean = static_cast<const float *>(a.mean), *rstd = static_cast<const float *>(a.rstd);
    const int C = a.C;
    const int64_t extent = a.N * C;
    const float inv_C = 1.0f / (float)C;
    float dw[KV][VEC], db[KV][VEC];
    bool held[KV];                       // the thread has channels of this vector
#pragma unroll
    for (int k = 0; k < KV; ++k) {
        held[k] = (k * threads + t) * VEC < C;
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[k][i] = db[k][i] = 0.0f;
    }
    const int64_t warp_first = G == 0 ? first : (int64_t)blockIdx.x * (blockDim.x / G) + (threadIdx.x & ~31) / (G == 0 ? 1 : G);

    Raw<T, VEC> rx[KV], rr[KV], rd[KV], re[KV];
    float mu = 0.0f, rs = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool valid = row < a.N && span_ok(a.err, row * C, C, extent);
        const int64_t base = row * C;
        mu = valid ? __ldg(mean + row) : 0.0f;
        rs = valid ? __ldg(rstd + row) : 0.0f;
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const int c = (k * threads + t) * VEC;
            const bool mine = valid && held[k];
            rx[k].zero(); rr[k].zero(); rd[k].zero(); re[k].zero();
            if (mine) {
                rx[k].load(x + base + c);
                rd[k].load(dy + base + c);
                if (res) rr[k].load(res + base + c);
                if (ds) re[k].load(ds + base + c);
            }
        }
    };
    fetch(first);
    for (int64_t row = first, lead = warp_first; lead < a.N; row += step, lead += step) {
        const bool valid = row < a.N;
        const int64_t base = row * C;
        const float m = mu, r = rs;
        float xh[KV][VEC], g[KV][VEC], e[KV][VEC];
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const int c = (k * threads + t) * VEC;
            rx[k].unpack(xh[k]);
            rd[k].unpack(g[k]);
            if (res) {
                rr[k].unpack(e[k]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) xh[k][i] += e[k][i];
            }
            if (ds) re[k].unpack(e[k]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                // a row past the end has m = r = 0 and grad_out 0: it adds nothing
                xh[k][i] = held[k] ? (xh[k][i] - m) * r : 0.0f;
                dw[k][i] = fmaf(g[k][i], xh[k][i], dw[k][i]);
                db[k][i] += g[k][i];
            }
            if (w && held[k]) {
                Raw<W, VEC> rw;
                float f[VEC];
                rw.load(w + c);
                rw.unpack(f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) g[k][i] *= f[i];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[0] += g[k][i];
                v[1] = fmaf(g[k][i], xh[k][i], v[1]);
            }
        }
        fetch(row + step);               // the next row's loads run under this row's sums
        row_sum<G>(v, &scratch, turn);
        const float c1 = v[0] * inv_C, c2 = v[1] * inv_C;
        if (dx) {
#pragma unroll
            for (int k = 0; k < KV; ++k) {
                const int c = (k * threads + t) * VEC;
                if (!valid || !held[k] || !span_ok(a.err, base + c, VEC, extent)) continue;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    o[i] = r * (g[k][i] - c1 - xh[k][i] * c2);
                    if (ds) o[i] += e[k][i];
                }
                Raw<T, VEC>::store(dx + base + c, o);
            }
        }
    }
    if (!a.partial) return;
    float *mine = a.partial + (int64_t)blockIdx.x * 2 * C;
    if (G == 0) {
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const int c = (k * threads + t) * VEC;
            if (!held[k]) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                mine[c + i] = dw[k][i];
                mine[C + c + i] = db[k][i];
            }
        }
        return;
    }
    // the block's groups: lanes of one warp with shuffles, warps through shared memory
#pragma unroll
    for (int k = 0; k < KV; ++k) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
            for (int off = G == 0 ? 32 : G; off < 32; off <<= 1) {
                dw[k][i] += __shfl_xor_sync(0xffffffffu, dw[k][i], off);
                db[k][i] += __shfl_xor_sync(0xffffffffu, db[k][i], off);
            }
        }
    }
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) < (G == 0 ? 32 : G)) {
        float *to = columns + (int64_t)warp * 2 * C;
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const int c = (k * threads + t) * VEC;
            if (!held[k]) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                to[c + i] = dw[k][i];
                to[C + c + i] = db[k][i];
            }
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * C; j += blockDim.x) {
        float v = 0.0f;
        for (int i = 0; i < warps; ++i) v += columns[i * 2 * C + j];
        mine[j] = v;
    }
}

// grad_weight and grad_bias from the blocks' partial sums: a block adds 32 of
// the 2*C columns, its warps every 32nd row of partials each, in a fixed order.
template <typename W, typename A>
__global__ void __launch_bounds__(1024) norm_columns_kernel(const A *partial, int rows, int C,
                                                            W *grad_weight, W *grad_bias) {
    __shared__ A part[32][33];
    cudaGridDependencySynchronize();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * 32 + tx, n = 2 * (int64_t)C;
    A v = 0;
    if (j < n) {
#pragma unroll 4
        for (int r = ty; r < rows; r += warps) v += partial[(int64_t)r * n + j];
    }
    part[ty][tx] = v;
    __syncthreads();
    if (ty != 0 || j >= n) return;
    v = 0;
    for (int i = 0; i < warps; ++i) v += part[i][tx];
    W *to = j < C ? grad_weight : grad_bias;
    if (!to) return;
    if constexpr (sizeof(W) == 8) to[j < C ? j : j - C] = v;
    else to[j < C ? j : j - C] = Elem<W>::from_f((float)v);
}

// ---------------------------------------------------------------- general
// Rows of any length and fp64: one kernel for grad_x (a block per row, two
// passes over it), one for the column sums (a thread per channel and chunk of
// rows).

template <typename T> struct BAcc { using type = float; };
template <> struct BAcc<double> { using type = double; };
template <typename T> __device__ __forceinline__ typename BAcc<T>::type up(T v) {
    if constexpr (sizeof(T) == 8) return v;
    else return Elem<T>::to_f(v);
}
template <typename T, typename A> __device__ __forceinline__ T down(A v) {
    if constexpr (sizeof(T) == 8) return v;
    else return Elem<T>::from_f((float)v);
}

template <typename T, typename W>
__global__ void __launch_bounds__(512) norm_backward_rows_general_kernel(const NormArgs a) {
    using A = typename BAcc<T>::type;
    __shared__ A scratch[2][kMaxWarps];
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const T *dy = static_cast<const T *>(a.grad_out), *ds = static_cast<const T *>(a.grad_sum);
    const W *w = static_cast<const W *>(a.weight);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const int64_t base = row * a.C;
        if (!span_ok(a.err, base, a.C, a.N * a.C)) continue;
        const A m = static_cast<const A *>(a.mean)[row], r = static_cast<const A *>(a.rstd)[row];
        A v0 = 0, v1 = 0;
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            const A s = up<T>(x[base + c]) + (res ? up<T>(res[base + c]) : (A)0);
            const A g = up<T>(dy[base + c]) * (w ? (A)up<W>(w[c]) : (A)1);
            v0 += g;
            v1 += g * ((s - m) * r);
        }
        for (int off = 16; off > 0; off >>= 1) {
            v0 += __shfl_xor_sync(0xffffffffu, v0, off);
            v1 += __shfl_xor_sync(0xffffffffu, v1, off);
        }
        __syncthreads();
        if (lane == 0) { scratch[0][warp] = v0; scratch[1][warp] = v1; }
        __syncthreads();
        v0 = v1 = 0;
        for (int i = 0; i < warps; ++i) { v0 += scratch[0][i]; v1 += scratch[1][i]; }
        const A c1 = v0 / (A)a.C, c2 = v1 / (A)a.C;
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            const A s = up<T>(x[base + c]) + (res ? up<T>(res[base + c]) : (A)0);
            const A g = up<T>(dy[base + c]) * (w ? (A)up<W>(w[c]) : (A)1);
            A o = r * (g - c1 - (s - m) * r * c2);
            if (ds) o += up<T>(ds[base + c]);
            static_cast<T *>(a.grad_x)[base + c] = down<T, A>(o);
        }
    }
}

// blockIdx.x: 128 channels; blockIdx.y: rows y, y + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(128) norm_backward_columns_general_kernel(const NormArgs a) {
    using A = typename BAcc<T>::type;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const T *dy = static_cast<const T *>(a.grad_out);
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= a.C) return;
    A dw = 0, db = 0;
    for (int64_t row = blockIdx.y; row < a.N; row += gridDim.y) {
        if (!span_ok(a.err, row * a.C + c, 1, a.N * a.C)) continue;
        const A m = static_cast<const A *>(a.mean)[row], r = static_cast<const A *>(a.rstd)[row];
        const A s = up<T>(x[row * a.C + c]) + (res ? up<T>(res[row * a.C + c]) : (A)0);
        const A g = up<T>(dy[row * a.C + c]);
        dw += g * ((s - m) * r);
        db += g;
    }
    A *mine = reinterpret_cast<A *>(a.partial) + (int64_t)blockIdx.y * 2 * a.C;
    mine[c] = dw;
    mine[a.C + c] = db;
}

// ---------------------------------------------------------------- launches

template <typename W, typename A>
static cudaError_t launch_columns(const NormArgs &a, int rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((2 * (int64_t)a.C + 31) / 32));
    cfg.blockDim = dim3(rows >= 64 ? 1024 : 256);
    cfg.stream = stream;
    // launched while the rows' kernel drains; the kernel waits for its results
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_columns_kernel<W, A>,
                              reinterpret_cast<const A *>(a.partial), rows, a.C,
                              static_cast<W *>(a.grad_weight), static_cast<W *>(a.grad_bias));
}

template <typename T, typename W>
static cudaError_t launch_general(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    using A = typename BAcc<T>::type;
    if (a.grad_x) {
        norm_backward_rows_general_kernel<T, W><<<(unsigned)(a.N < (1 << 20) ? a.N : (1 << 20)),
                                                  p.threads, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!a.partial) return cudaSuccess;
    const dim3 grid((unsigned)(((int64_t)a.C + 127) / 128), (unsigned)p.blocks);
    norm_backward_columns_general_kernel<T><<<grid, 128, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_columns<W, A>(a, p.blocks, stream);
}

template <typename T, typename W, int G, int KV, int VEC>
static cudaError_t launch_rows(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    const size_t smem = G == 0 || !a.partial ? 0 : (size_t)(p.threads / 32) * 2 * a.C * sizeof(float);
    static_assert(G == 0 || KV * VEC * G * 2 * 8 * 4 <= 48 * 1024, "columns fit the default shared memory");
    norm_backward_kernel<T, W, G, KV, VEC><<<p.blocks, p.threads, smem, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess || !a.partial ? e : launch_columns<W, float>(a, p.blocks, stream);
}

template <typename T, typename W>
static cudaError_t launch_backward_t(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
#define BWD(g, kv, vec) \
    if (p.G == g && p.KV == kv) return launch_rows<T, W, g, kv, vec>(a, p, stream);
    if (p.general) return launch_general<T, W>(a, p, stream);
    if (p.vec) {
        constexpr int V = Vec16<T>::N;
        BWD(4, 1, V) BWD(8, 1, V) BWD(16, 1, V) BWD(32, 1, V) BWD(32, 2, V)
        BWD(0, 1, V) BWD(0, 2, V) BWD(0, 4, V)
    } else {
        BWD(32, 1, 1) BWD(32, 4, 1) BWD(32, 8, 1) BWD(0, 4, 1) BWD(0, 8, 1)
    }
#undef BWD
    return cudaErrorInvalidValue;
}

cudaError_t launch_norm_backward(const NormArgs &a, const NormPlan &p, msda_dtype_t dt,
                                 msda_dtype_t pdt, cudaStream_t stream) {
    const bool wide = pdt == MSDA_F32;
    switch (dt) {
        case MSDA_F32: return launch_backward_t<float, float>(a, p, stream);
        case MSDA_BF16: return wide ? launch_backward_t<__nv_bfloat16, float>(a, p, stream)
                                    : launch_backward_t<__nv_bfloat16, __nv_bfloat16>(a, p, stream);
        case MSDA_F16: return wide ? launch_backward_t<__half, float>(a, p, stream)
                                   : launch_backward_t<__half, __half>(a, p, stream);
        case MSDA_F64: return launch_general<double, double>(a, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace msda
