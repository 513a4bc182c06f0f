// Layer norm's shared pieces: arguments, how a row is held and fetched, and
// sums over the threads that hold one row. The kernels are in
// msda_norm_forward.cu and msda_norm_backward.cu.
//
// A row of C channels lies in aligned 16-byte granules of V elements. It is
// held by a group of threads, KV granules each: thread t of g has granules t,
// t + g, ... of the row. A group is G = 2 to 32 lanes of one warp, or (G = 0)
// some whole warps of a block. A block holds several groups.
//
// Rows that do not start on 16-byte boundaries (RAGGED: C not a multiple of V)
// are held by the granules they touch: row r starts `phase` = r*C mod V
// elements into its first one, and the elements of a granule that belong to a
// neighbour are masked. A thread's rows are a multiple of V apart, so that its
// phase, and with it its channels, stay the same from row to row. That keeps
// the weights and the column sums of a thread in its registers.
#pragma once

#include "msda_common.cuh"

namespace msda {

constexpr int kSMs = 152;
// threads of a block whose rows are held by lanes of a warp: the backward's
// blocks are larger, since each leaves a row of partial sums
constexpr int kForwardThreads = 128, kBackwardThreads = 256;
// dynamic shared memory a launch may ask for without raising the kernel's
// limit: 48 KB less what the kernels declare themselves
constexpr size_t kDefaultShared = 47 * 1024;

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
    unsigned *err;                 // checked build: device word of range faults
};

// How a problem's rows are held, chosen on the host.
struct NormPlan {
    bool general;      // the looping kernels: fp64, rows past the registers, odd pointers
    bool ragged;
    int G, KV;
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

// V parameters of type W at w as fp32 pairs; `fill` where w is NULL.
template <typename W, int V>
__device__ __forceinline__ void load_params(float2 *v, const W *w, int c, float fill) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[i] = both(fill);
        return;
    }
    const uint4 *p = reinterpret_cast<const uint4 *>(w + c);
    constexpr int per = Vec16<W>::N;
#pragma unroll
    for (int i = 0; i < V / per; ++i) unpack_pairs<W>(v + i * per / 2, ldg16(p + i));
}
// The same for a masked granule: element by element, `fill` outside [0, C).
template <typename W, int V>
__device__ __forceinline__ void load_params_masked(float2 *v, const W *w, int c, int C, float fill) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const int a = c + 2 * i, b = a + 1;
        v[i].x = w && a >= 0 && a < C ? Elem<W>::to_f(w[a]) : fill;
        v[i].y = w && b >= 0 && b < C ? Elem<W>::to_f(w[b]) : fill;
    }
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
template <int R> struct BlockScratch { float v[2][R][kMaxWarps]; };

template <int G, int R>
__device__ __forceinline__ void row_sum(float (&v)[R], BlockScratch<R> *scratch, int &turn, int group,
                                        int index) {
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

// The place of a thread among the rows and of its granules in them. TH: threads
// of a block whose rows are held by lanes of a warp.
template <int G, int KV, int V, bool RAGGED, int TH> struct RowMap {
    int t, threads, index;         // of the group: this thread's place, its threads, its place in the block
    int64_t first, step, lead;     // the thread's rows; the first row of its warp
    int phase, granules;           // granules a row of this phase touches
    __device__ __forceinline__ RowMap(const NormArgs &a) {
        const int C = a.C;
        threads = G == 0 ? a.group : G;
        index = threadIdx.x / threads;
        t = threadIdx.x - index * threads;
        const int per_block = G == 0 ? blockDim.x / threads : TH / threads;
        first = (int64_t)blockIdx.x * per_block + index;
        lead = G == 0 ? first : (int64_t)blockIdx.x * per_block + (threadIdx.x & ~31) / threads;
        step = (int64_t)gridDim.x * per_block;
        phase = RAGGED ? (int)((first & (V - 1)) * (C & (V - 1)) & (V - 1)) : 0;
        granules = (phase + C + V - 1) / V;
    }
    __device__ __forceinline__ int granule(int k) const { return k * threads + t; }
    __device__ __forceinline__ bool held(int k) const { return granule(k) < granules; }
    // the channel of granule k's element 0 (negative in a first granule shared with the row before)
    __device__ __forceinline__ int channel(int k) const { return granule(k) * V - phase; }
    // all of granule k's elements belong to the row
    __device__ __forceinline__ bool whole(int k, int C) const {
        return !RAGGED || (channel(k) >= 0 && channel(k) + V <= C);
    }
    __device__ __forceinline__ bool has(int k, int i, int C) const {
        return !RAGGED || (channel(k) + i >= 0 && channel(k) + i < C);
    }
    // element offset of the thread's first granule in the tensor: a multiple of V
    __device__ __forceinline__ int64_t start(int C) const { return first * C - phase + (int64_t)t * V; }
    // A store at element `at` that leaves the neighbours' elements of a shared granule alone.
    template <typename T>
    __device__ __forceinline__ void store(T *p, int64_t at, int k, int C, const float2 *v) const {
        T *to = p + at + k * threads * V;
        if (whole(k, C)) {
            *reinterpret_cast<uint4 *>(to) = pack_pairs<T>(v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (has(k, i, C)) to[i] = Elem<T>::from_f(i & 1 ? v[i / 2].y : v[i / 2].x);
        }
    }
    // Starts the copy of granule k of the row at element `at` into `to`. Where
    // the thread has no such granule, or the row is past the last (!there), the
    // slot gets zeros and nothing is read.
    template <typename T>
    __device__ __forceinline__ void fetch(uint4 *to, const T *p, int64_t at, int k, bool there, int64_t extent,
                                          unsigned *err) const {
        const int64_t off = at + k * threads * V;
        there = there && held(k);
        int n = RAGGED && off + V > extent ? (int)(extent - off) : V;
        if (there && !span_ok(err, off, n, extent)) there = false;
        fetch16(to, there ? p + off : p, there ? n * (int)sizeof(T) : 0);
    }
};

}  // namespace msda
