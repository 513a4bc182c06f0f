// Layer norm's shared pieces: arguments, how rows are held and fetched, and
// sums over the threads that hold one row. The kernels are in
// msda_norm_forward.cuh and msda_norm_backward.cuh, in three forms:
//
// rows   Rows that all start on 16-byte boundaries. A row lies in 16-byte
//        granules of V elements and is held by a group of threads, KV granules
//        each: thread t of g has granules t, t + g, ... A thread fetches what
//        it will read itself.
// tiles  Rows that start anywhere (C not a multiple of V, or a tensor off a
//        16-byte boundary). Consecutive rows are one span of memory: a block
//        fetches the granules a few rows touch into shared memory and its
//        groups read their rows from there element by element, thread t having
//        channels t, t + g, ..., E of them; the results go back the same way.
// general  Rows of any length, in loops over memory: fp64, and rows too long
//        for the registers.
//
// A group is G = 2 to 32 lanes of one warp, or (G = 0) some whole warps of a
// block; a block holds several groups.
#pragma once

#include "msda_common.cuh"

namespace msda {

constexpr int kSMs = 152;
// threads of a block whose groups are lanes of a warp: rows form, tiles form
constexpr int kGroupThreads = 128, kTileThreads = 256;
// dynamic shared memory a launch may ask for without raising the kernel's
// limit: 48 KB less what the kernels declare themselves
constexpr size_t kDefaultShared = 47 * 1024;
// the limit it is raised to, always the same: two host threads that launch one
// kernel with different sizes must not lower each other's
constexpr int kRaisedShared = 226 * 1024;

struct NormArgs {
    const void *x, *residual;      // (N, C); residual NULL: none
    const void *weight, *bias;     // (C,) of the parameter type; NULL: ones / zeros
    void *out, *sum;               // (N, C); sum NULL: not wanted
    void *mean, *rstd;             // (N,) float (double for fp64); forward NULL: not wanted
    const void *grad_out, *grad_sum;   // backward; grad_sum NULL: none
    void *grad_x, *grad_weight, *grad_bias;
    float *partial;                // backward: (blocks, 2, C) sums of the column gradients
    double eps;
    int64_t N;
    int C;
    int group;                     // threads of a group of warps (G = 0)
    // tiles: rows of a group in a tile; tiles under way in shared memory, 2, or 1
    // where two do not fit
    int tile_rows, stages;
    unsigned *err;                 // checked build: device word of range faults
    // sums that the workspace has room for (last: between the pointers it cost the
    // backward of 8192 x 1024 bf16 2%)
    int64_t partials;
};

// How a problem's rows are held, chosen on the host.
struct NormPlan {
    enum Form { kRows, kTiles, kGeneral } form;
    int G, KV;                     // KV: granules (rows) or pairs of channels (tiles) of a thread
    int group, threads, blocks;    // threads of a group and of a block
};

// Checked build: the span [off, off + n) of a tensor of `extent` elements (see
// in_tensor); always true in the normal build.
__device__ __forceinline__ bool span_ok(unsigned *err, int64_t off, int64_t n, int64_t extent) {
#ifdef MSDA_CHECKED
    const bool ok = off >= 0 && n >= 0 && off <= extent - n;
    if (!ok && err) atomicOr(err, 1u);
    return ok;
#else
    return true;
#endif
}

// ------------------------------------------------- packed pairs of fp32
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <typename T> __device__ __forceinline__ void unpack_pairs(float2 *v, uint4 raw) {
    float f[Vec16<T>::N];
    unpack16<T>(f, raw);
#pragma unroll
    for (int i = 0; i < Vec16<T>::N / 2; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}
template <> __device__ __forceinline__ void unpack_pairs<__half>(float2 *v, uint4 raw) {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
}
template <typename T> __device__ __forceinline__ uint4 pack_pairs(const float2 *v) {
    float f[Vec16<T>::N];
#pragma unroll
    for (int i = 0; i < Vec16<T>::N / 2; ++i) {
        f[2 * i] = v[i].x;
        f[2 * i + 1] = v[i].y;
    }
    return pack16<T>(f);
}

// Parameters c to c + V of type W, of C at w, as fp32 pairs; `fill` where w is NULL.
template <typename W, int V>
__device__ __forceinline__ void load_params(float2 *v, const W *w, int c, float fill, int C, unsigned *err) {
    if (!w || !span_ok(err, c, V, C)) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[i] = both(fill);
        return;
    }
    const uint4 *p = reinterpret_cast<const uint4 *>(w + c);
    constexpr int per = Vec16<W>::N;
#pragma unroll
    for (int i = 0; i < V / per; ++i) unpack_pairs<W>(v + i * per / 2, ldg16(p + i));
}
// ------------------------------------------------------------- row fetches
// Asynchronous 16-byte copy of a granule to shared memory; `bytes` < 16 reads
// only that many and fills the rest with zeros.
__device__ __forceinline__ void fetch16(uint4 *to, const void *from, int bytes) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void fetch_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Sums of two values over the lanes of a group of W: the first exchange leaves
// one value to each half, so that a pair costs little more than a single one.
template <int W> __device__ __forceinline__ void lanes_sum2(float &a, float &b) {
    if constexpr (W == 1) return;
    const bool high = threadIdx.x & (W / 2);
    float v = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, W / 2);
#pragma unroll
    for (int off = W / 4; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const float w = __shfl_xor_sync(0xffffffffu, v, W / 2);
    a = high ? w : v;
    b = high ? v : w;
}
template <int W> __device__ __forceinline__ void lanes_sum(float &a) {
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
}

// Sums of R = 1 or 2 values over the threads of one row, the result in each of
// them. Groups of warps (G = 0) pass through shared memory with one barrier of
// their own: `turn` alternates two buffers, so that a warp that is ahead cannot
// overwrite values still being read.
constexpr int kMaxWarps = 16;
struct BlockScratch { float v[2][2][kMaxWarps]; };

template <int G, int R>
__device__ __forceinline__ void row_sum(float (&v)[R], BlockScratch *scratch, int &turn, int group, int index) {
    constexpr int W = G == 0 ? 32 : G;
    if constexpr (R == 2) lanes_sum2<W>(v[0], v[1]);
    else lanes_sum<W>(v[0]);
    if constexpr (G == 0) {
        const int lane = threadIdx.x & 31, warps = group >> 5, lead = index * warps;
        if (lane < R) scratch->v[turn][lane][threadIdx.x >> 5] = R == 2 && lane == 1 ? v[R - 1] : v[0];
        asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(group) : "memory");
        const bool mine = (lane & 15) < warps;
        if constexpr (R == 2) {          // lanes 0-15 add one value, lanes 16-31 the other
            float u = mine ? scratch->v[turn][lane >> 4][lead + (lane & 15)] : 0.0f;
            lanes_sum<16>(u);
            const float w = __shfl_xor_sync(0xffffffffu, u, 16);
            v[0] = lane < 16 ? u : w;
            v[1] = lane < 16 ? w : u;
        } else {
            v[0] = mine ? scratch->v[turn][0][lead + (lane & 15)] : 0.0f;
            lanes_sum<16>(v[0]);
        }
        turn ^= 1;
    }
}

// 1 / sqrt of a row's variance and eps, within 2 ulp; NaN where the squares left fp32's
// range (eps may: rstd is 0 then).
__device__ __forceinline__ float row_rstd(float squares, float inv_C, float eps) {
    return rsqrtf(fmaf(squares, inv_C, eps)) + (squares - squares);
}

// A row's mean is off by the roundings of its sum, up to 28 of them, and rstd
// multiplies these: a row of 10000.1 throughout would come out as -0.3. The distances
// from it add up to C times what it lacks. The quotient is corrected by its own
// remainder, so that an exact one comes out exact: in a row of equal entries every
// distance is the same multiple j <= 28 of one step, the sums of j and j^2 over up to
// 16,384 channels are exact below 2^24, and the shift is that distance and the sum of
// the squares about the corrected mean 0.
struct MeanFix { float shift, squares; };
__device__ __forceinline__ MeanFix fix_mean(float sum, float squares, float C, float inv_C) {
    float shift = sum * inv_C;
    shift = fmaf(fmaf(-shift, C, sum), inv_C, shift);
    squares = fmaf(-shift, sum, squares);
    return {shift, squares < 0.0f ? 0.0f : squares};     // NaN stays
}

// Where that is not done for every row (kFixAll), it is for rows whose mean is more than
// kFar / rstd; in others, whose entries' mean size is within (1 + kFar) / rstd, the
// mean's roundings are at most 28 * 2^-24 * (1 + kFar) of a normalised row (C / 512 + 26
// roundings in the general form). v: the variance and eps. (Zeros, infinities and NaN
// are far.)
constexpr float kFar = 2.0f;
template <typename A> __device__ __forceinline__ bool is_far(A mean, A v) {
    return !(mean * mean < (A)(kFar * kFar) * v);
}

// Rows form: groups of warps, which wait for their sums anyway, and fp32 rows fix every
// mean (86,016 x 256 fp32 40.8 us, 42.6 the other way; 8192 x 4096 bf16 45.0 us, 49.5),
// lanes with 16-bit rows those of far rows (44,446 x 256 bf16 11.8 us, 12.0; without any
// fix 11.3). The tiles and general forms, which issue or add what they wait for, the far
// ones (20,011 x 777 fp16 26.1 us, 28.4; without 25.3).
template <typename T, int G> constexpr bool kFixAll = G == 0 || sizeof(T) == 4;

// The place of a thread among the rows. TH: threads of a block whose groups are
// lanes of a warp.
template <int G, int TH> struct RowMap {
    int t, threads, index;         // of the group: this thread's place, its threads, its place in the block
    int rows;                      // of a block at a time: its groups
    int64_t first, step, lead;     // the thread's rows; the first row of its warp
    __device__ __forceinline__ RowMap(const NormArgs &a) {
        threads = G == 0 ? a.group : G;
        index = threadIdx.x / threads;
        t = threadIdx.x - index * threads;
        rows = (G == 0 ? blockDim.x : TH) / threads;
        first = (int64_t)blockIdx.x * rows + index;
        lead = G == 0 ? first : (int64_t)blockIdx.x * rows + (threadIdx.x & ~31) / threads;
        step = (int64_t)gridDim.x * rows;
    }
};

// The granules of a thread in its row (the rows form).
template <int G, int V, int TH> struct GranuleMap : RowMap<G, TH> {
    using RowMap<G, TH>::t;
    using RowMap<G, TH>::threads;
    using RowMap<G, TH>::first;
    int granules;
    __device__ __forceinline__ GranuleMap(const NormArgs &a) : RowMap<G, TH>(a), granules(a.C / V) {}
    __device__ __forceinline__ bool held(int k) const { return k * threads + t < granules; }
    __device__ __forceinline__ int channel(int k) const { return (k * threads + t) * V; }
    // element offset of the thread's first granule in the tensor
    __device__ __forceinline__ int64_t start(int C) const { return first * C + (int64_t)t * V; }
    template <typename T>
    __device__ __forceinline__ void store(T *p, int64_t at, int k, const float2 *v, int64_t extent,
                                          unsigned *err) const {
        if (span_ok(err, at + k * threads * V, V, extent))
            *reinterpret_cast<uint4 *>(p + at + k * threads * V) = pack_pairs<T>(v);
    }
    // Starts the copy of granule k of the row at element `at` into `to`. Where
    // the thread has no such granule, or the row is past the last (!there), the
    // slot gets zeros and nothing is read.
    template <typename T>
    __device__ __forceinline__ void fetch(uint4 *to, const T *p, int64_t at, int k, bool there, int64_t extent,
                                          unsigned *err) const {
        const int64_t off = at + k * threads * V;
        there = there && held(k) && span_ok(err, off, V, extent);
        fetch16(to, there ? p + off : p, there ? 16 : 0);
    }
};

// ------------------------------------------------------------------- tiles
// Spans of a tensor's elements by the granules they touch: `lead(at)` elements
// of the first granule come before the span.
constexpr int kTileE = 16;               // channels of a thread, at most, but for the longest rows (32)
template <typename T> struct Spans {
    static constexpr int V = Vec16<T>::N;
    T *base;
    int64_t extent;
    int phase;
    __device__ __forceinline__ Spans(const void *tensor, int64_t extent)
        : base(static_cast<T *>(const_cast<void *>(tensor))), extent(extent),
          phase((int)(reinterpret_cast<uintptr_t>(tensor) / sizeof(T)) & (V - 1)) {}
    __device__ __forceinline__ int lead(int64_t at) const { return (int)((unsigned)phase + (unsigned)at) & (V - 1); }
    // Starts the copies of the granules of n elements from `at` into shared
    // memory. Elements of them outside the tensor are not read.
    __device__ __forceinline__ void fetch(uint4 *to, int64_t at, int n, unsigned *err) const {
        const int l = lead(at), granules = (l + n + V - 1) / V;
        const int64_t from = at - l;
        const T *p = base + from;
        if (from >= 0 && from + granules * V <= extent) {
            if (!span_ok(err, from, granules * V, extent)) return;
            for (int i = threadIdx.x; i < granules; i += blockDim.x) fetch16(to + i, p + i * V, 16);
            return;
        }
        for (int i = threadIdx.x; i < granules; i += blockDim.x) {      // the tensor's first or last tile
            const int64_t off = from + i * V, left = extent - off;
            const int m = left < V ? (int)left : V;
            if (off >= 0) {
                if (span_ok(err, off, m, extent)) fetch16(to + i, p + i * V, m * (int)sizeof(T));
            } else {
                for (int k = (int)-off; k < m; ++k) reinterpret_cast<T *>(to + i)[k] = p[i * V + k];
            }
        }
    }
    // Writes n elements from `at` out of shared memory: whole granules, and
    // one by one the elements of a first and last that neighbours share.
    __device__ __forceinline__ void store(const uint4 *from, int64_t at, int n, unsigned *err) const {
        if (!span_ok(err, at, n, extent)) return;
        const int l = lead(at), end = l + n, first = l ? 1 : 0, last = end / V;
        T *p = base + (at - l);
        const T *e = reinterpret_cast<const T *>(from);
        for (int i = first + threadIdx.x; i < last; i += blockDim.x) reinterpret_cast<uint4 *>(p)[i] = from[i];
        const int head = l + (int)threadIdx.x, tail = last * V + (int)threadIdx.x;
        if (l && head < V && head < end) p[head] = e[head];
        if (last >= first && tail < end) p[tail] = e[tail];
    }
};
// 16-byte places that any span of n elements fits.
template <typename T> constexpr __host__ __device__ int tile_places(int64_t n) {
    return (int)((n + 2 * Vec16<T>::N - 2) / Vec16<T>::N);
}

// The tiles that fit beside `outs` results: two, or one, of `ins` tensors each.
constexpr size_t kMostShared = 220 * 1024;
constexpr int tile_stages(int ins, int outs, size_t bytes) {
    return (size_t)(2 * ins + outs) * bytes <= kMostShared ? 2 : 1;
}

// Rows of a group in a tile: up to four, in tiles of up to 16 KB, or of 32 KB where
// a block has an SM to itself and two tiles fit (3,661 x 4097 bf16 backward: 58 us
// with 16 KB, 49 so); two at least, while the blocks an SM can hold keep their
// tiles (31,128 x 257 fp32 forward: 20.1 us with one, 16.8 so); and as many as
// leave every block its tile. More rows a tile share its copies' and barriers' cost.
inline int tile_rows(const NormArgs &a, const NormPlan &p, int ins, int outs, int bytes) {
    const int64_t one = (int64_t)(p.threads / p.group) * a.C * bytes;
    const int64_t resident = p.threads > 256 ? 1 : 512 / p.threads;
    int64_t n = (p.threads > 256 && tile_stages(ins, outs, 33 * 1024) == 2 ? 32 * 1024 : 16 * 1024) / one;
    if (n < 2 && resident * (2 * ins + outs) * (2 * one + 32) <= (int64_t)kMostShared) n = 2;
    const int64_t share = a.N / ((int64_t)p.blocks * (p.threads / p.group));
    const int64_t most = share < 4 ? (share < 1 ? 1 : share) : 4;
    return (int)(n < 1 ? 1 : n < most ? n : most);
}

// A thread's channels t, t + g, ... as P pairs: pair i is channels t + 2i*g and
// t + (2i + 1)*g. The group's size is such that all but the last two of six or
// eight pairs lie in the row, half of sixteen and none of four; only the others
// look at each channel. There are no branches around pairs: they would keep the
// shared memory's reads apart.
template <int P> constexpr int kWholePairs = P == 4 ? 0 : P == 16 ? 8 : P - 2;
// With sixteen pairs a thread's registers do not hold its weights beside them.
template <int P> constexpr bool kHoldsWeights = P <= 8;
template <typename T, bool WHOLE>
__device__ __forceinline__ float2 load_pair(const T *row, int c, int g, int C) {
    if constexpr (WHOLE) return make_float2(Elem<T>::to_f(row[c]), Elem<T>::to_f(row[c + g]));
    return make_float2(c < C ? Elem<T>::to_f(row[c]) : 0.0f, c + g < C ? Elem<T>::to_f(row[c + g]) : 0.0f);
}
template <int P, typename T>
__device__ __forceinline__ void load_pairs(float2 (&v)[P], const T *row, int t, int g, int C) {
    constexpr int W = kWholePairs<P>;
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = load_pair<T, true>(row, t + 2 * i * g, g, C);
#pragma unroll
    for (int i = W; i < P; ++i) v[i] = load_pair<T, false>(row, t + 2 * i * g, g, C);
}
// Checked build: the pairs taken to lie in the row do.
template <int P> __device__ __forceinline__ bool pairs_ok(unsigned *err, int t, int g, int C) {
    return kWholePairs<P> == 0 || span_ok(err, t + (2 * kWholePairs<P> - 1) * g, 1, C);
}
template <int P, typename W>
__device__ __forceinline__ void load_weights(float2 (&v)[P], const W *w, int t, int g, int C, float fill,
                                             unsigned *err) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = both(fill);
    if (w && pairs_ok<P>(err, t, g, C)) load_pairs(v, w, t, g, C);
}
template <int P, typename T>
__device__ __forceinline__ void store_pairs(T *row, int t, int g, int C, const float2 (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = t + 2 * i * g;
        if (i < kWholePairs<P> || c < C) row[c] = Elem<T>::from_f(v[i].x);
        if (i < kWholePairs<P> || c + g < C) row[c + g] = Elem<T>::from_f(v[i].y);
    }
}

}  // namespace msda
