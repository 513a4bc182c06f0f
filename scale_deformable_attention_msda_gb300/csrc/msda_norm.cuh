// Layer norm's shared pieces: arguments, vector access, and sums over the
// threads that hold one row. The kernels are in msda_norm_forward.cu and
// msda_norm_backward.cu.
//
// A row of C channels is held by G threads, KV vectors of VEC channels each
// (channel (k*G + t)*VEC + i belongs to thread t). VEC is 16 bytes' worth
// where every row starts on a 16-byte boundary, and 1 otherwise. G is 4 to 32
// lanes of one warp, or (G = 0) a whole block.
#pragma once

#include "msda_common.cuh"

namespace msda {

constexpr int kSMs = 152;

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
    unsigned *err;                 // checked build: device word of range faults
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

// N elements of T as fp32, in 16-byte accesses (VEC > 1) or one element.
template <typename T, int VEC> struct Raw {
    static constexpr int kWords = VEC * (int)sizeof(T) / 16;
    uint4 w[kWords];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = ldg16(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void unpack(float *v) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) unpack16<T>(v + i * Vec16<T>::N, w[i]);
    }
    static __device__ __forceinline__ void store(T *p, const float *v) {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            reinterpret_cast<uint4 *>(p)[i] = pack16<T>(v + i * Vec16<T>::N);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
};
template <typename T> struct Raw<T, 1> {
    T e;
    __device__ __forceinline__ void load(const T *p) { e = *p; }
    __device__ __forceinline__ void unpack(float *v) const { v[0] = Elem<T>::to_f(e); }
    static __device__ __forceinline__ void store(T *p, const float *v) { *p = Elem<T>::from_f(v[0]); }
    __device__ __forceinline__ void zero() { e = Elem<T>::from_f(0.0f); }
};

// Sums of R values over the threads of one row, the result in each of them.
// Block rows (G = 0) pass through shared memory with one barrier: `turn`
// alternates two buffers, so that a warp that is ahead cannot overwrite values
// still being read.
constexpr int kMaxWarps = 32;
template <int R> struct BlockScratch { float v[2][R][kMaxWarps]; };

template <int G, int R>
__device__ __forceinline__ void row_sum(float (&v)[R], BlockScratch<R> *scratch, int &turn) {
    constexpr int W = G == 0 ? 32 : G;
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) {
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], off);
    }
    if (G == 0) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        if (lane == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) scratch->v[turn][r][warp] = v[r];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = lane < warps ? scratch->v[turn][r][lane] : 0.0f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], off);
        }
        turn ^= 1;
    }
}

// How a problem's rows are held, chosen on the host.
struct NormPlan {
    bool general;      // the looping kernels (fp64, and rows past the registers)
    bool vec;          // 16-byte vectors
    int G, KV;         // threads per row (0: a block) and vectors per thread
    int threads;       // of a block
    int blocks;
};

}  // namespace msda
