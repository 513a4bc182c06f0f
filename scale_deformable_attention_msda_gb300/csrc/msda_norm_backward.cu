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

// S: rows whose copies are under way while one is worked on. A thread copies
// what it reads itself, so its own wait is all the order the copies need.
template <typename T, typename W, int G, int KV, bool RAGGED, int S, int TH>
__global__ void __launch_bounds__(TH) norm_backward_kernel(const NormArgs a) {
    constexpr int V = Vec16<T>::N, P = V / 2;
    __shared__ BlockScratch<2> scratch;
    extern __shared__ uint4 ring[];      // (S, tensors, KV, threads); at the end (warps, 2, C) floats
    int turn = 0;
    cudaTriggerProgrammaticLaunchCompletion();   // the column kernel may be launched; it waits for this one's end
    const int C = a.C;
    const RowMap<G, KV, V, RAGGED, TH> map(a);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const T *dy = static_cast<const T *>(a.grad_out), *ds = static_cast<const T *>(a.grad_sum);
    const W *w = static_cast<const W *>(a.weight);
    T *dx = static_cast<T *>(a.grad_x);
    const float *mean = static_cast<const float *>(a.mean), *rstd = static_cast<const float *>(a.rstd);
    const int64_t extent = a.N * C, hop = map.step * C;
    const float inv_C = 1.0f / (float)C;
    const int plane = G == 0 ? blockDim.x : TH;   // a thread's slots are this far apart
    const int tensors = 2 + (res ? 1 : 0) + (ds ? 1 : 0), tall = tensors * KV * plane;
    const int ds_at = (tensors - 1) * KV;
    int64_t here = map.start(C), ahead = here;
    int64_t coming = map.first;          // the row at `ahead`
    auto fetch = [&](uint4 *to) {
        const bool there = coming < a.N;
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            map.fetch(to + k * plane, x, ahead, k, there, extent, a.err);
            map.fetch(to + (KV + k) * plane, dy, ahead, k, there, extent, a.err);
            if (res) map.fetch(to + (2 * KV + k) * plane, res, ahead, k, there, extent, a.err);
            if (ds) map.fetch(to + (ds_at + k) * plane, ds, ahead, k, there, extent, a.err);
        }
        coming += map.step;
        ahead += hop;
        fetch_commit();
    };
    uint4 *const begin = ring + threadIdx.x, *slot = begin;
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(begin + i * tall);
    float2 pw[KV][P], dw[KV][P], db[KV][P];
#pragma unroll
    for (int k = 0; k < KV; ++k) {
#pragma unroll
        for (int i = 0; i < P; ++i) dw[k][i] = db[k][i] = both(0.0f);
        if (RAGGED) load_params_masked<W, V>(pw[k], w, map.channel(k), C, 1.0f);
        else load_params<W, V>(pw[k], map.held(k) ? w : nullptr, map.channel(k), 1.0f);
    }
    float mu = 0.0f, rs = 0.0f;
    if (map.first < a.N) {
        mu = __ldg(mean + map.first);
        rs = __ldg(rstd + map.first);
    }
    for (int64_t row = map.first, lead = map.lead; lead < a.N; row += map.step, lead += map.step, here += hop) {
        // a row past the last, and a granule the thread does not have, were
        // filled with zeros: grad_out = 0 there, and nothing is added
        const bool valid = G == 0 || G == 32 || row < a.N;
        const float m = mu, r = rs;
        if (row + map.step < a.N) {
            mu = __ldg(mean + row + map.step);
            rs = __ldg(rstd + row + map.step);
        }
        float2 xh[KV][P], g[KV][P];
        float2 v0 = both(0.0f), v1 = both(0.0f);
        fetch_wait<S - 1>();
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            unpack_pairs<T>(xh[k], slot[k * plane]);
            unpack_pairs<T>(g[k], slot[(KV + k) * plane]);
            if (res) {
                float2 e[P];
                unpack_pairs<T>(e, slot[(2 * KV + k) * plane]);
#pragma unroll
                for (int i = 0; i < P; ++i) xh[k][i] = add2(xh[k][i], e[i]);
            }
            if (RAGGED && !map.whole(k, C)) {      // a neighbour's elements: s = mean, grad_out = 0
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if (!map.has(k, 2 * i, C)) { xh[k][i].x = m; g[k][i].x = 0.0f; }
                    if (!map.has(k, 2 * i + 1, C)) { xh[k][i].y = m; g[k][i].y = 0.0f; }
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                xh[k][i] = mul2(add2(xh[k][i], both(-m)), both(r));
                dw[k][i] = fma2(g[k][i], xh[k][i], dw[k][i]);
                db[k][i] = add2(db[k][i], g[k][i]);
                g[k][i] = mul2(g[k][i], pw[k][i]);
                v0 = add2(v0, g[k][i]);
                v1 = fma2(g[k][i], xh[k][i], v1);
            }
        }
        float v[2] = {v0.x + v0.y, v1.x + v1.y};
        row_sum<G>(v, &scratch, turn, map.threads, map.index);
        if (dx) {
            const float2 c1 = both(-v[0] * inv_C), c2 = both(-v[1] * inv_C);
#pragma unroll
            for (int k = 0; k < KV; ++k) {
                float2 e[P];
                if (ds) unpack_pairs<T>(e, slot[(ds_at + k) * plane]);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    g[k][i] = mul2(fma2(xh[k][i], c2, add2(g[k][i], c1)), both(r));
                    if (ds) g[k][i] = add2(g[k][i], e[i]);
                }
                if (valid && map.held(k)) map.store(dx, here, k, C, g[k]);
            }
        }
        fetch(slot);
        slot = slot + tall == begin + S * tall ? begin : slot + tall;
    }
    fetch_wait<0>();
    if (!a.partial) return;
    // the block's sums: each group leaves its own in shared memory, or, where
    // all rows have the same phase, each warp after adding its groups' sums
    constexpr bool FOLD = !RAGGED && G > 0 && G < 32;
    if constexpr (FOLD) {
#pragma unroll
        for (int k = 0; k < KV; ++k) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
#pragma unroll
                for (int off = G; off < 32; off <<= 1) {
                    dw[k][i].x += __shfl_xor_sync(0xffffffffu, dw[k][i].x, off);
                    dw[k][i].y += __shfl_xor_sync(0xffffffffu, dw[k][i].y, off);
                    db[k][i].x += __shfl_xor_sync(0xffffffffu, db[k][i].x, off);
                    db[k][i].y += __shfl_xor_sync(0xffffffffu, db[k][i].y, off);
                }
            }
        }
    }
    __syncthreads();                     // the ring's space is used again
    float *columns = reinterpret_cast<float *>(ring);
    const int writer = FOLD ? threadIdx.x >> 5 : map.index;
    const int writers = FOLD ? blockDim.x >> 5 : blockDim.x / map.threads;
    if (!FOLD || (threadIdx.x & 31) < G) {
        float *to = columns + writer * 2 * C;
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            if (!map.held(k)) continue;
            const int c = map.channel(k);
            if constexpr (!RAGGED) {
#pragma unroll
                for (int i = 0; i < P / 2; ++i) {
                    reinterpret_cast<float4 *>(to + c)[i] =
                        make_float4(dw[k][2 * i].x, dw[k][2 * i].y, dw[k][2 * i + 1].x, dw[k][2 * i + 1].y);
                    reinterpret_cast<float4 *>(to + C + c)[i] =
                        make_float4(db[k][2 * i].x, db[k][2 * i].y, db[k][2 * i + 1].x, db[k][2 * i + 1].y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (!map.has(k, i, C)) continue;
                    to[c + i] = i & 1 ? dw[k][i / 2].y : dw[k][i / 2].x;
                    to[C + c + i] = i & 1 ? db[k][i / 2].y : db[k][i / 2].x;
                }
            }
        }
    }
    __syncthreads();
    float *mine = a.partial + (int64_t)blockIdx.x * 2 * C;
    for (int j = threadIdx.x; j < 2 * C; j += blockDim.x) {
        float v = 0.0f;
        for (int i = 0; i < writers; ++i) v += columns[i * 2 * C + j];
        mine[j] = v;
    }
}

// grad_weight and grad_bias from the blocks' partial sums, added in a fixed
// order: a block takes TW of the 2*C columns, its threads every
// (threads / TW)th row of partials each. TW = 8 (one 32-byte sector) spreads
// few channels over more SMs; the rows' reads are what it waits for.
template <typename W, typename A, int TW>
__global__ void __launch_bounds__(1024) norm_columns_kernel(const A *partial, int rows, int C,
                                                            W *grad_weight, W *grad_bias) {
    __shared__ A part[32][TW];
    cudaGridDependencySynchronize();
    const int tx = threadIdx.x % TW, ty = threadIdx.x / TW, step = blockDim.x / TW;
    const int64_t j = (int64_t)blockIdx.x * TW + tx;
    const bool mine = j < 2 * (int64_t)C;
    const int64_t c = j < C ? j : j - C;
    A v = 0;
    if (mine) {
#pragma unroll 8
        for (int r = ty; r < rows; r += step) v += partial[r * 2 * (int64_t)C + j];
    }
#pragma unroll
    for (int off = TW; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) < TW) part[threadIdx.x >> 5][tx] = v;
    __syncthreads();
    if (threadIdx.x >= TW || !mine) return;
    v = 0;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += part[i][tx];
    W *to = j < C ? grad_weight : grad_bias;
    if (!to) return;
    if constexpr (sizeof(W) == 8) to[c] = v;
    else to[c] = Elem<W>::from_f((float)v);
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
    const bool narrow = a.C < 2048;
    const int tw = narrow ? 8 : 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((2 * (int64_t)a.C + tw - 1) / tw));
    cfg.blockDim = dim3(rows >= 8 * 1024 / tw ? 1024 : rows >= 2 * 1024 / tw ? 512 : 256);
    cfg.stream = stream;
    // launched while the rows' kernel runs; the kernel waits for its results
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, narrow ? norm_columns_kernel<W, A, 8> : norm_columns_kernel<W, A, 32>,
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

template <typename T, typename W, int G, int KV, bool RAGGED, int S, int TH>
static cudaError_t launch_rows(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    auto kernel = norm_backward_kernel<T, W, G, KV, RAGGED, S, TH>;
    const int tensors = 2 + (a.residual ? 1 : 0) + (a.grad_sum ? 1 : 0);
    size_t smem = (size_t)S * tensors * KV * p.threads * 16;
    if (a.partial) {
        const int writers = G > 0 && !RAGGED ? p.threads / 32 : p.threads / p.group;
        const size_t columns = (size_t)writers * 2 * a.C * sizeof(float);
        smem = smem > columns ? smem : columns;
    }
    if (smem > kDefaultShared) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.blocks, p.threads, smem, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess || !a.partial ? e : launch_columns<W, float>(a, p.blocks, stream);
}

template <typename T, typename W>
static cudaError_t launch_backward_t(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
#define BWD(g, kv, r, s) \
    if (p.G == g && p.KV == kv && p.ragged == r) return launch_rows<T, W, g, kv, r, s, g == 0 ? 512 : kBackwardThreads>(a, p, stream);
    if (p.general) return launch_general<T, W>(a, p, stream);
#ifdef NORM_TUNE
    NORM_TUNE
#else
    BWD(2, 2, false, 2) BWD(4, 2, false, 2) BWD(8, 2, false, 2) BWD(16, 2, false, 2) BWD(32, 2, false, 2)
    BWD(0, 2, false, 2) BWD(0, 4, false, 1)
    BWD(2, 2, true, 2) BWD(4, 2, true, 2) BWD(8, 2, true, 2) BWD(16, 2, true, 2) BWD(32, 2, true, 2)
    BWD(0, 2, true, 2) BWD(0, 4, true, 1)
#endif
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
