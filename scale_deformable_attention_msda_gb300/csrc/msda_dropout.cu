// Dropout from a counter-based generator: the mask is a function of the entry's
// number, the draw's number and the seed, computed where it is used and never
// stored (contract in include/msda.h).
//
// What bounds it: memory, 4 bytes an entry for 16-bit data without a residual.
// The generator runs beside: Philox4x32-10 has 20 wide products for 128 bits. At
// 32 bits an entry these alone would take as long as the copy of 16-bit data; at
// 16 bits an entry, which tells probabilities 2^-16 apart, they take half of it.
#include <math.h>

#include "msda_common.cuh"
#include "msda_host.h"

namespace msda {
namespace {

constexpr int kThreads = 256;

struct DropArgs {
    const void *x, *residual;
    void *out;
    const int64_t *counter;
    int64_t n;
    uint32_t threshold;
    double factor;
};

struct Philox {
    uint32_t w[4];
    __device__ __forceinline__ Philox(int64_t seed, int64_t number, int64_t block) {
        uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)((uint64_t)seed >> 32);
        w[0] = (uint32_t)block;
        w[1] = (uint32_t)((uint64_t)block >> 32);
        w[2] = (uint32_t)number;
        w[3] = (uint32_t)((uint64_t)number >> 32);
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t a = (uint64_t)w[0] * 0xD2511F53u, b = (uint64_t)w[2] * 0xCD9E8D57u;
            w[0] = (uint32_t)(b >> 32) ^ w[1] ^ k0;
            w[1] = (uint32_t)b;
            w[2] = (uint32_t)(a >> 32) ^ w[3] ^ k1;
            w[3] = (uint32_t)a;
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
    }
    // 16 bits of entry e of the eight
    __device__ __forceinline__ uint32_t half(int e) const { return e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu; }
};

template <typename T> struct Wide { using type = float; };
template <> struct Wide<double> { using type = double; };
template <typename T> __device__ __forceinline__ typename Wide<T>::type widen(T v) { return Elem<T>::to_f(v); }
template <> __device__ __forceinline__ double widen<double>(double v) { return v; }
template <typename T> __device__ __forceinline__ T narrow(typename Wide<T>::type v) { return Elem<T>::from_f(v); }
template <> __device__ __forceinline__ double narrow<double>(double v) { return v; }

// 16 bytes that are read once, asked for where this stands: before the generator's rounds.
__device__ __forceinline__ uint4 fetch(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <typename T> union Eight {
    static constexpr int P = 8 * sizeof(T) / 16;
    uint4 raw[P];
    T v[8];
    __device__ Eight() {}
};

// The eight entries of one call of the generator.
template <typename T, bool RES>
__device__ __forceinline__ void drop_eight(Eight<T> &in, const Eight<T> &add, const DropArgs &a, int64_t seed, int64_t number, int64_t i) {
    using W = typename Wide<T>::type;
    const W factor = (W)a.factor;
    const Philox r(seed, number, i);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const W kept = r.half(j) >= a.threshold ? widen<T>(in.v[j]) * factor : (W)0;
        in.v[j] = narrow<T>(RES ? kept + widen<T>(add.v[j]) : kept);
    }
}

// VEC: all tensors start on 16-byte boundaries, and a thread has 32 bytes of each under
// way. The last entries, and all without VEC, go one by one.
template <typename T, bool VEC> constexpr int kAtOnce = VEC && sizeof(T) == 2 ? 2 : 1;
template <typename T, bool VEC, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropArgs a) {
    constexpr int AT_ONCE = kAtOnce<T, VEC>, P = Eight<T>::P;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    T *out = static_cast<T *>(a.out);
    const int64_t seed = a.counter[0], number = a.counter[1], whole = VEC ? a.n / 8 : 0, blocks = (a.n + 7) / 8;
    const int64_t step = (int64_t)gridDim.x * kThreads, first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    for (int64_t i = first; i < blocks; i += AT_ONCE * step) {
        Eight<T> in[AT_ONCE], add[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int64_t at = i + u * step;
            if (at >= whole) continue;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                in[u].raw[j] = fetch(reinterpret_cast<const uint4 *>(x + 8 * at) + j);
                if (RES) add[u].raw[j] = fetch(reinterpret_cast<const uint4 *>(res + 8 * at) + j);
            }
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int64_t at = i + u * step;
            if (at < whole) {
                drop_eight<T, RES>(in[u], add[u], a, seed, number, at);
#pragma unroll
                for (int j = 0; j < P; ++j) reinterpret_cast<uint4 *>(out + 8 * at)[j] = in[u].raw[j];
            } else if (at < blocks) {
                const int many = a.n - 8 * at < 8 ? (int)(a.n - 8 * at) : 8;
                Eight<T> one, other;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < many) {
                        one.v[j] = x[8 * at + j];
                        if (RES) other.v[j] = res[8 * at + j];
                    }
                drop_eight<T, RES>(one, other, a, seed, number, at);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < many) out[8 * at + j] = one.v[j];
            }
        }
    }
}

__global__ void dropout_next_kernel(int64_t *state, int64_t *drawn) {
    drawn[0] = state[0];
    drawn[1] = (int64_t)atomicAdd(reinterpret_cast<unsigned long long *>(state + 1), 1ull);
}

template <typename T> cudaError_t launch(const DropArgs &a, cudaStream_t stream) {
    const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                       reinterpret_cast<uintptr_t>(a.out)) % 16) == 0;
    const int64_t per = (int64_t)kThreads * (vec ? kAtOnce<T, true> : 1), want = ((a.n + 7) / 8 + per - 1) / per, cap = (int64_t)1 << 30;
    const unsigned blocks = (unsigned)(want < cap ? want : cap);
    if (vec && a.residual) dropout_kernel<T, true, true><<<blocks, kThreads, 0, stream>>>(a);
    else if (vec) dropout_kernel<T, true, false><<<blocks, kThreads, 0, stream>>>(a);
    else if (a.residual) dropout_kernel<T, false, true><<<blocks, kThreads, 0, stream>>>(a);
    else dropout_kernel<T, false, false><<<blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace msda

extern "C" {

msda_status_t msda_dropout(const void *x, const void *residual, void *out, int64_t n, double p,
                           const int64_t *counter, msda_dtype_t dtype, void *stream) {
    if (dtype != MSDA_F32 && dtype != MSDA_BF16 && dtype != MSDA_F16 && dtype != MSDA_F64) return MSDA_ERR_DTYPE;
    if (n < 0 || n > ((int64_t)1 << 60) || !(p >= 0.0 && p <= 1.0)) return MSDA_ERR_SHAPE;
    if (n == 0) return MSDA_OK;
    if (!x || !out || !counter) return MSDA_ERR_NULL;
    const uintptr_t e = dtype == MSDA_F64 ? 8 : dtype == MSDA_F32 ? 4 : 2;
    if (!msda::aligned(x, e) || !msda::aligned(residual, e) || !msda::aligned(out, e) || !msda::aligned(counter, 8))
        return MSDA_ERR_ALIGN;
    msda::DropArgs a = {x, residual, out, counter, n, 0u, 0.0};
    a.threshold = (uint32_t)nearbyint(p * 65536.0);
    a.factor = a.threshold < 65536u ? 65536.0 / (65536.0 - a.threshold) : 0.0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err = dtype == MSDA_F32  ? msda::launch<float>(a, s)
                          : dtype == MSDA_BF16 ? msda::launch<__nv_bfloat16>(a, s)
                          : dtype == MSDA_F16  ? msda::launch<__half>(a, s)
                                               : msda::launch<double>(a, s);
    return err == cudaSuccess ? MSDA_OK : MSDA_ERR_CUDA;
}

msda_status_t msda_dropout_next(int64_t *state, int64_t *drawn, void *stream) {
    if (!state || !drawn) return MSDA_ERR_NULL;
    if (!msda::aligned(state, 8) || !msda::aligned(drawn, 8)) return MSDA_ERR_ALIGN;
    msda::dropout_next_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(state, drawn);
    return cudaGetLastError() == cudaSuccess ? MSDA_OK : MSDA_ERR_CUDA;
}

}  // extern "C"
