// Layer norm, backward. With xh = (s - mean) * rstd and g = grad_out * weight,
//
//   grad_x      = rstd * (g - mean_c(g) - xh * mean_c(g * xh)) + grad_sum
//   grad_weight = sum over the rows of grad_out * xh
//   grad_bias   = sum over the rows of grad_out
//
// One pass: while a row is in registers its threads add its part of the column
// sums to fp32 registers of their own (a thread keeps the same channels for all
// its rows). A block adds its threads' sums in shared memory and leaves one row of
// partial sums, and a second kernel, launched while the first runs, adds those in
// a fixed order. No atomics: results do not vary. A block that is alone writes the
// gradients itself.
//
// What bounds it: memory and issue about evenly. 44,446 rows of 256 bf16 channels
// with a residual take 18.2 us, the second kernel's 3 us among them (5.0 TB/s of
// the data alone, 74% of the copy rate; the rows' kernel executes 181 warp
// instructions a row); 86,016 x 256 fp32 54.7 us (6.4 TB/s); 8192 x 4096 bf16 with both
// gradients 56.5 us (5.9 TB/s); 20,011 x 777 fp16, whose rows start anywhere, 38 us.
// The longest rows, 32 channels a thread, are bound by spills: 666 x 12,000 fp32 43.9
// us (2.2 TB/s; 1.1 million spill requests). 512 threads of an SM are what 128 registers each allow; with copies that hold no
// registers they keep about 60 KB on the way. (GB300, calls in a graph, inputs
// larger than L2.)
#pragma once

#include "msda_norm.cuh"

namespace msda {

// Sum over the lanes of a warp that hold the same channels.
template <int G> __device__ __forceinline__ float2 fold(float2 v) {
#pragma unroll
    for (int off = G; off < 32; off <<= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
    }
    return v;
}

// The block's row of partial sums from those its writers left in shared memory;
// a block that is the only one writes the gradients.
template <typename W>
__device__ __forceinline__ void leave_partials(const NormArgs &a, const float *columns, int writers) {
    __syncthreads();
    const int n = 2 * a.C;
    auto column = [&](int j) {
        float v = columns[j];
        for (int i = 1; i < writers; ++i) v += columns[i * n + j];
        return v;
    };
    if (gridDim.x > 1) {
        if (!span_ok(a.err, (int64_t)blockIdx.x * n, n, a.partials)) return;
        float *mine = a.partial + (int64_t)blockIdx.x * n;
#pragma unroll 4
        for (int j = threadIdx.x; j < n; j += blockDim.x) mine[j] = column(j);
        return;
    }
    W *gw = static_cast<W *>(a.grad_weight), *gb = static_cast<W *>(a.grad_bias);
    for (int j = threadIdx.x; j < a.C; j += blockDim.x) {
        if (gw) gw[j] = Elem<W>::from_f(column(j));
        if (gb) gb[j] = Elem<W>::from_f(column(a.C + j));
    }
}

// The rows form: see msda_norm.cuh. S: rows whose copies are under way while one
// is worked on. A thread copies what it reads itself, so its own wait is all the
// order the copies need.
template <typename T, typename W, int G, int KV, int S, int TH>
__global__ void __launch_bounds__(TH) norm_backward_kernel(const NormArgs a) {
    constexpr int V = Vec16<T>::N, P = V / 2;
    __shared__ BlockScratch scratch;
    extern __shared__ uint4 ring[];      // (S, tensors, KV, threads); at the end (warps, 2, C) floats
    int turn = 0;
    cudaTriggerProgrammaticLaunchCompletion();   // the column kernel may be launched; it waits for this one's end
    const int C = a.C;
    const GranuleMap<G, V, TH> map(a);
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
        load_params<W, V>(pw[k], map.held(k) ? w : nullptr, map.channel(k), 1.0f, C, a.err);
    }
    float mu = 0.0f, rs = 0.0f;
    if (map.first < a.N && span_ok(a.err, map.first, 1, a.N)) {
        mu = __ldg(mean + map.first);
        rs = __ldg(rstd + map.first);
    }
    for (int64_t row = map.first, lead = map.lead; lead < a.N; row += map.step, lead += map.step, here += hop) {
        // A row past the last, and a granule the thread does not have, were
        // filled with zeros: grad_out = 0 there, and with a mean of zero xh as
        // well, so that nothing is added. (Of a mean as it is, mean * rstd may
        // leave fp32's range, and 0 * inf is NaN.)
        const bool valid = G == 0 || G == 32 || row < a.N;
        const float m = mu, r = rs;
        mu = rs = 0.0f;
        if (row + map.step < a.N && span_ok(a.err, row + map.step, 1, a.N)) {
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
            const float from = map.held(k) ? -m : 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                xh[k][i] = mul2(add2(xh[k][i], both(from)), both(r));
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
                if (valid && map.held(k)) map.store(dx, here, k, g[k], extent, a.err);
            }
        }
        fetch(slot);
        slot = slot + tall == begin + S * tall ? begin : slot + tall;
    }
    fetch_wait<0>();
    if (!a.partial) return;
    // the block's sums: each group of warps leaves its own in shared memory,
    // and each warp after adding its lanes' groups
    constexpr bool FOLD = G > 0;
    if constexpr (FOLD) {
#pragma unroll
        for (int k = 0; k < KV; ++k) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                dw[k][i] = fold<G>(dw[k][i]);
                db[k][i] = fold<G>(db[k][i]);
            }
        }
    }
    __syncthreads();                     // the ring's space is used again
    float *columns = reinterpret_cast<float *>(ring);
    if (!FOLD || (threadIdx.x & 31) < G) {
        float *to = columns + (FOLD ? threadIdx.x >> 5 : map.index) * 2 * C;
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            if (!map.held(k)) continue;
            const int c = map.channel(k);
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
                reinterpret_cast<float4 *>(to + c)[i] =
                    make_float4(dw[k][2 * i].x, dw[k][2 * i].y, dw[k][2 * i + 1].x, dw[k][2 * i + 1].y);
                reinterpret_cast<float4 *>(to + C + c)[i] =
                    make_float4(db[k][2 * i].x, db[k][2 * i].y, db[k][2 * i + 1].x, db[k][2 * i + 1].y);
            }
        }
    }
    leave_partials<W>(a, columns, FOLD ? blockDim.x >> 5 : map.rows);
}

// The tiles form: see msda_norm.cuh.
template <typename T, typename W, int G, int P>
__global__ void __launch_bounds__(G == 0 ? 512 : kTileThreads, G == 0 ? 1 : 2)
norm_backward_tile_kernel(const NormArgs a) {
    constexpr int TH = kTileThreads;
    __shared__ BlockScratch scratch;
    extern __shared__ uint4 ring[];      // stages of (tensors, places), then grad_x; at the end (writers, 2, C) floats
    int turn = 0;
    cudaTriggerProgrammaticLaunchCompletion();
    const int C = a.C;
    const RowMap<G, TH> map(a);
    const int g = map.threads, t = map.t;
    const W *w = static_cast<const W *>(a.weight);
    const float *mean = static_cast<const float *>(a.mean), *rstd = static_cast<const float *>(a.rstd);
    const int64_t extent = a.N * C;
    const float inv_C = 1.0f / (float)C;
    const int tensors = 2 + (a.residual ? 1 : 0) + (a.grad_sum ? 1 : 0);
    const int rows = map.rows * a.tile_rows, places = tile_places<T>((int64_t)rows * C);
    uint4 *const outs = ring + a.stages * tensors * places;
    const Spans<T> xs(a.x, extent), ys(a.grad_out, extent), rs(a.residual, extent), ds(a.grad_sum, extent),
        os(a.grad_x, extent);
    const int ds_at = (tensors - 1) * places;
    const int64_t step = (int64_t)gridDim.x * rows;
    (void)pairs_ok<P>(a.err, t, g, C);
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.N) {
            uint4 *to = ring + stage * tensors * places;
            const int n = (int)(a.N - row < rows ? a.N - row : rows) * C;
            xs.fetch(to, row * C, n, a.err);
            ys.fetch(to + places, row * C, n, a.err);
            if (a.residual) rs.fetch(to + 2 * places, row * C, n, a.err);
            if (a.grad_sum) ds.fetch(to + ds_at, row * C, n, a.err);
        }
        fetch_commit();
    };
    const int64_t begin = (int64_t)blockIdx.x * rows;
    fetch(begin, 0);
    if (a.stages == 2) fetch(begin + step, 1);
    float2 pw[P], dw[P], db[P];
    load_weights(pw, w, t, g, C, 1.0f, a.err);
#pragma unroll
    for (int i = 0; i < P; ++i) dw[i] = db[i] = both(0.0f);
    int stage = 0;
    for (int64_t tile = begin; tile < a.N; tile += step) {
        const int64_t at = tile * C;
        const int there = (int)(a.N - tile < rows ? a.N - tile : rows);
        float m = 0.0f, r = 0.0f;        // of the group's next row
        if (map.index < there && span_ok(a.err, tile + map.index, 1, a.N)) {
            m = __ldg(mean + tile + map.index);
            r = __ldg(rstd + tile + map.index);
        }
        if (a.stages == 2) fetch_wait<1>();
        else fetch_wait<0>();
        __syncthreads();
        const uint4 *in = ring + stage * tensors * places;
        const T *x0 = reinterpret_cast<const T *>(in) + xs.lead(at);
        const T *y0 = reinterpret_cast<const T *>(in + places) + ys.lead(at);
        const T *r0 = reinterpret_cast<const T *>(in + 2 * places) + rs.lead(at);
        const T *d0 = reinterpret_cast<const T *>(in + ds_at) + ds.lead(at);
        T *o0 = reinterpret_cast<T *>(outs) + os.lead(at);
        // groups take the tile's rows in turn; all make the same number of turns
        for (int lead = 0; lead < there; lead += map.rows) {
            const int row = lead + map.index, from = row * C;
            const bool valid = row < there;
            const float mu = m, rstd_row = r;
            if (row + map.rows < there && span_ok(a.err, tile + row + map.rows, 1, a.N)) {
                m = __ldg(mean + tile + row + map.rows);
                r = __ldg(rstd + tile + row + map.rows);
            }
            float2 xh[P], gy[P];
            float2 v0 = both(0.0f), v1 = both(0.0f);
            if (valid) {
                load_pairs(xh, x0 + from, t, g, C);
                if (a.residual) {
                    float2 e[P];
                    load_pairs(e, r0 + from, t, g, C);
#pragma unroll
                    for (int i = 0; i < P; ++i) xh[i] = add2(xh[i], e[i]);
                }
                load_pairs(gy, y0 + from, t, g, C);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    // past the row grad_out is zero, and xh too
                    const int c = t + 2 * i * g;
                    const bool whole = i < kWholePairs<P>;
                    const float2 from = make_float2(whole || c < C ? -mu : 0.0f, whole || c + g < C ? -mu : 0.0f);
                    xh[i] = mul2(add2(xh[i], from), both(rstd_row));
                    dw[i] = fma2(gy[i], xh[i], dw[i]);
                    db[i] = add2(db[i], gy[i]);
                    gy[i] = mul2(gy[i], pw[i]);
                    v0 = add2(v0, gy[i]);
                    v1 = fma2(gy[i], xh[i], v1);
                }
            }
            float v[2] = {v0.x + v0.y, v1.x + v1.y};
            row_sum<G>(v, &scratch, turn, g, map.index);
            if (valid && a.grad_x) {
                const float2 c1 = both(-v[0] * inv_C), c2 = both(-v[1] * inv_C);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    gy[i] = mul2(fma2(xh[i], c2, add2(gy[i], c1)), both(rstd_row));
                if (a.grad_sum) {
                    load_pairs(xh, d0 + from, t, g, C);
#pragma unroll
                    for (int i = 0; i < P; ++i) gy[i] = add2(gy[i], xh[i]);
                }
                store_pairs(o0 + from, t, g, C, gy);
            }
        }
        __syncthreads();                 // the results are whole, the inputs used
        fetch(tile + a.stages * step, stage);
        stage ^= a.stages - 1;
        if (a.grad_x) os.store(outs, at, there * C, a.err);
    }
    fetch_wait<0>();
    if (!a.partial) return;
    constexpr bool FOLD = G > 0;
    if constexpr (FOLD) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            dw[i] = fold<G>(dw[i]);
            db[i] = fold<G>(db[i]);
        }
    }
    __syncthreads();                     // the tiles' space is used again
    float *columns = reinterpret_cast<float *>(ring);
    if (!FOLD || (threadIdx.x & 31) < G) {
        float *to = columns + (FOLD ? threadIdx.x >> 5 : map.index) * 2 * C;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = t + 2 * i * g;
            if (c < C) { to[c] = dw[i].x; to[C + c] = db[i].x; }
            if (c + g < C) { to[c + g] = dw[i].y; to[C + c + g] = db[i].y; }
        }
    }
    leave_partials<W>(a, columns, FOLD ? blockDim.x >> 5 : map.rows);
}

// grad_weight and grad_bias from the blocks' partial sums, added in a fixed
// order: a block takes TW of the 2*C columns, its threads every
// (threads / TW)th row of partials each. TW = 8 (one 32-byte sector) spreads
// few channels over more SMs; the rows' reads are what it waits for.
template <typename W, typename A, int TW>
__global__ void __launch_bounds__(1024) norm_columns_kernel(const A *partial, int64_t partials, int rows, int C,
                                                            W *grad_weight, W *grad_bias, unsigned *err) {
    __shared__ A part[32][TW];
    cudaGridDependencySynchronize();
    const int tx = threadIdx.x % TW, ty = threadIdx.x / TW, step = blockDim.x / TW;
    const int64_t j = (int64_t)blockIdx.x * TW + tx;
    const bool mine = j < 2 * (int64_t)C;
    const int64_t c = j < C ? j : j - C;
    A v = 0;
    if (mine && span_ok(err, (int64_t)(rows - 1) * 2 * C + j, 1, partials)) {
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
    if (!span_ok(a.err, (int64_t)blockIdx.y * 2 * a.C + c, a.C + 1, a.partials)) return;
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
                              reinterpret_cast<const A *>(a.partial), a.partials, rows, a.C,
                              static_cast<W *>(a.grad_weight), static_cast<W *>(a.grad_bias), a.err);
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

template <typename W>
static cudaError_t launch(void (*kernel)(const NormArgs), const NormArgs &a, const NormPlan &p, size_t smem,
                          cudaStream_t stream) {
    if (a.partial) {
        const int writers = p.G > 0 ? p.threads / 32 : p.threads / p.group;
        const size_t columns = (size_t)writers * 2 * a.C * sizeof(float);
        smem = smem > columns ? smem : columns;
    }
    if (smem > kDefaultShared) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRaisedShared);
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.blocks, p.threads, smem, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess || !a.partial || p.blocks == 1 ? e : launch_columns<W, float>(a, p.blocks, stream);
}

template <typename T, typename W, int G, int KV, int S, int TH>
static cudaError_t launch_rows(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    const int tensors = 2 + (a.residual ? 1 : 0) + (a.grad_sum ? 1 : 0);
    return launch<W>(norm_backward_kernel<T, W, G, KV, S, TH>, a, p, (size_t)S * tensors * KV * p.threads * 16,
                     stream);
}

template <typename T, typename W, int G, int P>
static cudaError_t launch_tiles(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    const int ins = 2 + (a.residual ? 1 : 0) + (a.grad_sum ? 1 : 0);
    NormArgs b = a;
    b.tile_rows = tile_rows(a, p, ins, 1, sizeof(T));
    const size_t bytes = (size_t)tile_places<T>((int64_t)(p.threads / p.group) * b.tile_rows * a.C) * 16;
    b.stages = tile_stages(ins, 1, bytes);
    return launch<W>(norm_backward_tile_kernel<T, W, G, P>, b, p, (b.stages * ins + 1) * bytes, stream);
}

template <typename T, typename W>
static cudaError_t launch_backward_t(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
#define ROWS(g, kv) \
    if (p.G == g && p.KV == kv) return launch_rows<T, W, g, kv, 2, g == 0 ? 512 : kGroupThreads>(a, p, stream);
#define TILES(g, pairs) \
    if (p.G == g && p.KV == pairs) return launch_tiles<T, W, g, pairs>(a, p, stream);
    if (p.form == NormPlan::kRows) {
        ROWS(2, 2) ROWS(4, 2) ROWS(8, 2) ROWS(16, 2) ROWS(32, 2) ROWS(32, 3)
        if constexpr (sizeof(T) == 4) {
            ROWS(2, 3) ROWS(4, 3) ROWS(8, 3) ROWS(16, 3) ROWS(32, 4)
            if (p.threads <= 384) { ROWS(0, 4) }
            if (p.G == 0 && p.KV == 8) return launch_rows<T, W, 0, 8, 1, 512>(a, p, stream);
        } else {
            ROWS(0, 2)
        }
        // the longest rows: one row's copies are what fits
        if (p.G == 0 && p.KV == 4) return launch_rows<T, W, 0, 4, 1, 512>(a, p, stream);
    } else if (p.form == NormPlan::kTiles) {
        TILES(2, 4) TILES(2, 6) TILES(2, 8) TILES(4, 6) TILES(4, 8) TILES(8, 6) TILES(8, 8) TILES(16, 6) TILES(16, 8)
        TILES(32, 6) TILES(32, 8) TILES(0, 6) TILES(0, 8)
    } else {
        return launch_general<T, W>(a, p, stream);
    }
#undef ROWS
#undef TILES
    return cudaErrorInvalidValue;
}

}  // namespace msda
