// Layer norm, forward: out = (s - mean) * rstd * weight + bias over the C
// channels of each row of s = x + residual, mean and biased variance per row.
//
// A row is read once and stays in registers: its mean, then the sum of squared
// distances from that mean (no difference of large sums), a correction of the mean
// by what the distances add up to (fix_mean in msda_norm.cuh), then the output. All
// arithmetic in fp32; s is not rounded before it is normalised, and out is rounded
// once.
//
// What bounds it: memory, where rows start on 16-byte boundaries. 44,446 rows of
// 256 bf16 channels with a residual take 11.7 us (5.8 TB/s, 86% of the copy rate);
// 86,016 x 256 fp32 40.9 us (6.5 TB/s); 8192 x 4096 bf16 with a residual and the
// sum 44.6 us (6.0 TB/s). Rows that start anywhere are bound by instructions, an
// element at a time from shared memory: 20,011 x 777 fp16 take 26.0 us (2.4 TB/s;
// 801 warp instructions a row). A few rows are bound by the launch: 300 x 256
// 1.8 us, one row of 8192 3.3 us. (GB300, calls in a graph, inputs larger than L2.
// Pairs of figures below that compare two forms or sizes were measured before means
// were corrected, which added up to 5%.)
#pragma once

#include "msda_norm.cuh"

namespace msda {

// The rows form: see msda_norm.cuh. S: rows whose copies are under way while one
// is worked on. A thread copies what it reads itself, so its own wait is all the
// order the copies need, and the copies hold no registers: with plain loads the
// same rows took 18.3 us instead of 11.2. Sums run on packed pairs of fp32, which
// take 10% fewer instructions than scalar ones. The bounds keep the blocks on an SM
// that the kernels had before their means were corrected: 4 with three or four
// granules, 5 or 6 with two.
template <typename T, typename W, int G, int KV, int S, int TH>
__global__ void __launch_bounds__(TH, G == 0 ? 1 : KV > 2 ? 4 : sizeof(T) == 4 ? 6 : 5)
norm_forward_kernel(const NormArgs a) {
    constexpr int V = Vec16<T>::N, P = V / 2;
    __shared__ BlockScratch scratch;
    extern __shared__ uint4 ring[];      // (S, tensors, KV, threads)
    int turn = 0;
    const int C = a.C;
    const GranuleMap<G, V, TH> map(a);
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
        load_params<W, V>(pw[k], map.held(k) ? w : nullptr, c, 1.0f, C, a.err);
        load_params<W, V>(pb[k], map.held(k) ? b : nullptr, c, 0.0f, C, a.err);
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
            if (a.sum && valid && map.held(k)) map.store(static_cast<T *>(a.sum), here, k, s[k], extent, a.err);
#pragma unroll
            for (int i = 0; i < P; ++i) acc = add2(acc, s[k][i]);
        }
        float v[1] = {acc.x + acc.y};
        row_sum<G>(v, &scratch, turn, map.threads, map.index);
        fetch(slot);
        slot = slot + tall == begin + S * tall ? begin : slot + tall;
        const float mean = v[0] * inv_C;
        float shift = 0.0f, squares;
        float2 off = both(0.0f);
        acc = both(0.0f);
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            const float m = map.held(k) ? -mean : 0.0f;      // a slot without a granule stays zero
#pragma unroll
            for (int i = 0; i < P; ++i) s[k][i] = add2(s[k][i], both(m));
#pragma unroll
            for (int i = 0; i < P; ++i) acc = fma2(s[k][i], s[k][i], acc);
            if constexpr (kFixAll<T, G>) {
#pragma unroll
                for (int i = 0; i < P; ++i) off = add2(off, s[k][i]);
            }
        }
        if constexpr (kFixAll<T, G>) {
            float u[2] = {off.x + off.y, acc.x + acc.y};
            row_sum<G>(u, &scratch, turn, map.threads, map.index);
            const MeanFix f = fix_mean(u[0], u[1], (float)C, inv_C);
            shift = f.shift;
            squares = f.squares;
        } else {
            v[0] = acc.x + acc.y;
            row_sum<G>(v, &scratch, turn, map.threads, map.index);
            squares = v[0];
            const bool far = is_far(mean, fmaf(squares, inv_C, (float)a.eps));
            if (__any_sync(0xffffffffu, far)) {      // the same for a group's lanes
#pragma unroll
                for (int k = 0; k < KV; ++k) {
#pragma unroll
                    for (int i = 0; i < P; ++i) off = add2(off, s[k][i]);
                }
                float u[1] = {off.x + off.y};
                row_sum<G>(u, &scratch, turn, map.threads, map.index);
                const MeanFix f = fix_mean(u[0], squares, (float)C, inv_C);
                shift = far ? f.shift : 0.0f;
                squares = far ? f.squares : squares;
            }
        }
        const float rstd = row_rstd(squares, inv_C, (float)a.eps);
        if (map.t == 0 && valid && a.mean && span_ok(a.err, row, 1, a.N)) {
            static_cast<float *>(a.mean)[row] = mean + shift;
            static_cast<float *>(a.rstd)[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < KV; ++k) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                s[k][i] = fma2(mul2(add2(s[k][i], both(-shift)), both(rstd)), pw[k][i], pb[k][i]);
            if (valid && map.held(k)) map.store(static_cast<T *>(a.out), here, k, s[k], extent, a.err);
        }
    }
    fetch_wait<0>();
}

// The tiles form: see msda_norm.cuh.
template <typename T, typename W, int G, int P>
__global__ void __launch_bounds__(G == 0 ? 512 : kTileThreads, G == 0 ? 1 : 3)
norm_forward_tile_kernel(const NormArgs a) {
    constexpr int TH = kTileThreads;
    __shared__ BlockScratch scratch;
    extern __shared__ uint4 ring[];      // stages of (tensors, places), then out and sum
    int turn = 0;
    const int C = a.C;
    const RowMap<G, TH> map(a);
    const int g = map.threads, t = map.t;
    const W *w = static_cast<const W *>(a.weight), *b = static_cast<const W *>(a.bias);
    const int64_t extent = a.N * C;
    const float inv_C = 1.0f / (float)C;
    const int rows = map.rows * a.tile_rows;
    const int tensors = a.residual ? 2 : 1, places = tile_places<T>((int64_t)rows * C);
    uint4 *const outs = ring + a.stages * tensors * places;
    const Spans<T> xs(a.x, extent), rs(a.residual, extent), os(a.out, extent), ss(a.sum, extent);
    const int64_t step = (int64_t)gridDim.x * rows;
    (void)pairs_ok<P>(a.err, t, g, C);
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.N) {
            uint4 *to = ring + stage * tensors * places;
            const int n = (int)(a.N - row < rows ? a.N - row : rows) * C;
            xs.fetch(to, row * C, n, a.err);
            if (a.residual) rs.fetch(to + places, row * C, n, a.err);
        }
        fetch_commit();
    };
    const int64_t begin = (int64_t)blockIdx.x * rows;
    fetch(begin, 0);
    if (a.stages == 2) fetch(begin + step, 1);
    constexpr int HELD = kHoldsWeights<P> ? P : 1;
    float2 pw[HELD], pb[HELD];
    if constexpr (kHoldsWeights<P>) {
        load_weights(pw, w, t, g, C, 1.0f, a.err);
        load_weights(pb, b, t, g, C, 0.0f, a.err);
    }
    int stage = 0;
    for (int64_t tile = begin; tile < a.N; tile += step) {
        const int64_t at = tile * C;
        const int there = (int)(a.N - tile < rows ? a.N - tile : rows);
        if (a.stages == 2) fetch_wait<1>();
        else fetch_wait<0>();
        __syncthreads();
        const uint4 *in = ring + stage * tensors * places;
        const T *x0 = reinterpret_cast<const T *>(in) + xs.lead(at);
        const T *r0 = reinterpret_cast<const T *>(in + places) + rs.lead(at);
        T *o0 = reinterpret_cast<T *>(outs) + os.lead(at), *s0 = reinterpret_cast<T *>(outs + places) + ss.lead(at);
        // groups take the tile's rows in turn; all make the same number of turns
        for (int lead = 0; lead < there; lead += map.rows) {
            const int row = lead + map.index;
            const bool valid = row < there;
            const int from = (valid ? row : 0) * C;      // a group without a row repeats the first, unwritten
            float2 s[P], acc = both(0.0f);
            load_pairs(s, x0 + from, t, g, C);
            if (a.residual) {
                float2 e[P];
                load_pairs(e, r0 + from, t, g, C);
#pragma unroll
                for (int i = 0; i < P; ++i) s[i] = add2(s[i], e[i]);
            }
            if (a.sum && valid) store_pairs(s0 + from, t, g, C, s);
#pragma unroll
            for (int i = 0; i < P; ++i) acc = add2(acc, s[i]);
            float v[1] = {acc.x + acc.y};
            row_sum<G>(v, &scratch, turn, g, map.index);
            float mean = v[0] * inv_C;
            acc = both(0.0f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = t + 2 * i * g;
                const bool whole = i < kWholePairs<P>;
                s[i] = add2(s[i], make_float2(whole || c < C ? -mean : 0.0f, whole || c + g < C ? -mean : 0.0f));
                acc = fma2(s[i], s[i], acc);
            }
            v[0] = acc.x + acc.y;
            row_sum<G>(v, &scratch, turn, g, map.index);
            float squares = v[0];
            const bool far = is_far(mean, fmaf(squares, inv_C, (float)a.eps));
            if (G == 0 ? far : __any_sync(0xffffffffu, far)) {   // the same for a group's threads
                acc = both(0.0f);
#pragma unroll
                for (int i = 0; i < P; ++i) acc = add2(acc, s[i]);
                float u[1] = {acc.x + acc.y};
                row_sum<G>(u, &scratch, turn, g, map.index);
                if (far) {
                    const MeanFix f = fix_mean(u[0], squares, (float)C, inv_C);
                    squares = f.squares;
                    mean += f.shift;
#pragma unroll
                    for (int i = 0; i < P; ++i) s[i] = add2(s[i], both(-f.shift));
                }
            }
            if (!valid) continue;
            const float rstd = row_rstd(squares, inv_C, (float)a.eps);
            if (t == 0 && a.mean && span_ok(a.err, tile + row, 1, a.N)) {
                static_cast<float *>(a.mean)[tile + row] = mean;
                static_cast<float *>(a.rstd)[tile + row] = rstd;
            }
#pragma unroll
            for (int i = 0; i < P; ++i) s[i] = mul2(s[i], both(rstd));
            if constexpr (kHoldsWeights<P>) {
#pragma unroll
                for (int i = 0; i < P; ++i) s[i] = fma2(s[i], pw[i], pb[i]);
            } else {
                float2 e[P];
                load_weights(e, w, t, g, C, 1.0f, a.err);
#pragma unroll
                for (int i = 0; i < P; ++i) s[i] = mul2(s[i], e[i]);
                load_weights(e, b, t, g, C, 0.0f, a.err);
#pragma unroll
                for (int i = 0; i < P; ++i) s[i] = add2(s[i], e[i]);
            }
            store_pairs(o0 + from, t, g, C, s);
        }
        __syncthreads();                 // the outputs are whole, the inputs used
        fetch(tile + a.stages * step, stage);
        stage ^= a.stages - 1;
        os.store(outs, at, there * C, a.err);
        if (a.sum) ss.store(outs + places, at, there * C, a.err);
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

// Rows of any length, one block each, read three times (the later reads hit
// the caches), five times where the row is_far: then the mean is that of the
// distances from the row's first entry, so that a row of equal entries has exactly
// that mean, corrected by what the distances from it add up to. (fp64 additions are
// what 2000 x 1024 fp64 wait for: 201 us; with the correction in every row 294.)
template <typename T, typename W>
__global__ void __launch_bounds__(512) norm_forward_general_kernel(const NormArgs a) {
    using A = typename Acc<T>::type;
    __shared__ A scratch[kMaxWarps];
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const W *w = static_cast<const W *>(a.weight), *b = static_cast<const W *>(a.bias);
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const int64_t base = row * a.C;
        if (!span_ok(a.err, base, a.C, a.N * a.C)) continue;
        auto at = [&](int c) { return to_acc<T>(x[base + c]) + (res ? to_acc<T>(res[base + c]) : (A)0); };
        A v = 0, shift = 0;
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) v += at(c);
        A mean = block_sum<A>(v, scratch) / (A)a.C;
        v = 0;
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            const A d = at(c) - mean;
            v += d * d;
        }
        A squares = block_sum<A>(v, scratch);
        v = squares / (A)a.C + (A)a.eps;
        if (is_far(mean, v)) {                           // the same for all threads
            const A first = at(0);
            v = 0;
            for (int c = threadIdx.x; c < a.C; c += blockDim.x) v += at(c) - first;
            mean = first + block_sum<A>(v, scratch) / (A)a.C;
            A off = 0;
            v = 0;
            for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
                const A d = at(c) - mean;
                off += d;
                v += d * d;
            }
            off = block_sum<A>(off, scratch);
            shift = off / (A)a.C;
            squares = block_sum<A>(v, scratch) - shift * off;
            squares = squares < (A)0 ? (A)0 : squares;
            v = squares / (A)a.C + (A)a.eps;
        }
        const A rstd = (A)1 / sqrt(v) + (squares - squares);     // squares out of range: NaN
        if (threadIdx.x == 0 && a.mean) {
            static_cast<A *>(a.mean)[row] = mean + shift;
            static_cast<A *>(a.rstd)[row] = rstd;
        }
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            const A s = at(c);
            if (a.sum) static_cast<T *>(a.sum)[base + c] = from_acc<T, A>(s);
            A g = (s - mean - shift) * rstd;
            if (w) g *= (A)to_acc<W>(w[c]);
            if (b) g += (A)to_acc<W>(b[c]);
            static_cast<T *>(a.out)[base + c] = from_acc<T, A>(g);
        }
    }
}

// A launch with `smem` bytes of dynamic shared memory.
static cudaError_t launch(void (*kernel)(const NormArgs), const NormArgs &a, const NormPlan &p, size_t smem,
                          cudaStream_t stream) {
    if (smem > kDefaultShared) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRaisedShared);
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.blocks, p.threads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, typename W, int G, int KV, int S, int TH>
static cudaError_t launch_rows(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    return launch(norm_forward_kernel<T, W, G, KV, S, TH>, a, p,
                  (size_t)S * (a.residual ? 2 : 1) * KV * p.threads * 16, stream);
}

template <typename T, typename W, int G, int P>
static cudaError_t launch_tiles(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
    const int ins = a.residual ? 2 : 1, outs = a.sum ? 2 : 1;
    NormArgs b = a;
    b.tile_rows = tile_rows(a, p, ins, outs, sizeof(T));
    const size_t bytes = (size_t)tile_places<T>((int64_t)(p.threads / p.group) * b.tile_rows * a.C) * 16;
    b.stages = tile_stages(ins, outs, bytes);
    return launch(norm_forward_tile_kernel<T, W, G, P>, b, p, (b.stages * ins + outs) * bytes, stream);
}

template <typename T, typename W>
static cudaError_t launch_forward_t(const NormArgs &a, const NormPlan &p, cudaStream_t stream) {
#define ROWS(g, kv) \
    if (p.G == g && p.KV == kv) return launch_rows<T, W, g, kv, 2, kGroupThreads>(a, p, stream);
#define TILES(g, pairs) \
    if (p.G == g && p.KV == pairs) return launch_tiles<T, W, g, pairs>(a, p, stream);
    if (p.form == NormPlan::kRows) {
        ROWS(2, 2) ROWS(2, 3) ROWS(4, 2) ROWS(4, 3) ROWS(8, 2) ROWS(8, 3) ROWS(16, 2) ROWS(16, 3)
        ROWS(32, 2) ROWS(32, 3) ROWS(32, 4)
        if constexpr (sizeof(T) == 2) {
            if (p.G == 0 && p.KV == 2) return launch_rows<T, W, 0, 2, 2, 512>(a, p, stream);
        }
        if constexpr (sizeof(T) == 4) {
            if (p.G == 0 && p.KV == 8) return launch_rows<T, W, 0, 8, 1, 512>(a, p, stream);
        }
        // Four granules: two rows under way, or one row of two tensors (4096 x
        // 4096 fp32 with a residual and the sum: 41.8 us, two 43.1; 8000 x 1000
        // without: 12.5 us, two 11.4).
        if (p.G == 0 && p.KV == 4)
            return a.residual || p.threads > 448 ? launch_rows<T, W, 0, 4, 1, 512>(a, p, stream)
                                                 : launch_rows<T, W, 0, 4, 2, 512>(a, p, stream);
    } else if (p.form == NormPlan::kTiles) {
        TILES(2, 4) TILES(2, 6) TILES(2, 8) TILES(4, 6) TILES(4, 8) TILES(8, 6) TILES(8, 8) TILES(16, 6) TILES(16, 8)
        TILES(32, 6) TILES(32, 8) TILES(0, 6) TILES(0, 8) TILES(0, 16)
    } else {
        return launch(norm_forward_general_kernel<T, W>, a, p, 0, stream);
    }
#undef ROWS
#undef TILES
    return cudaErrorInvalidValue;
}

}  // namespace msda
