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
cudaError_t fault_word_for_launch(unsigned **err);
namespace {

constexpr int kThreads = 256;

struct DropArgs {
    const void *x, *residual;
    void *out;
    const int64_t *counter;
    int64_t n;
    uint32_t threshold;
    double factor;
    unsigned *err;
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

// Eight entries a thread and turn: one call of the generator. VEC: all tensors
// start on 16-byte boundaries.
template <typename T, bool VEC, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropArgs a) {
    using W = typename Wide<T>::type;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    T *out = static_cast<T *>(a.out);
    const int64_t seed = a.counter[0], number = a.counter[1], blocks = (a.n + 7) / 8;
    const W factor = (W)a.factor;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < blocks; i += (int64_t)gridDim.x * kThreads) {
        constexpr int P = 8 * sizeof(T) / 16;
        union Eight { uint4 raw[P]; T v[8]; __device__ Eight() {} } in, add;
        const int64_t at = 8 * i;
        const int many = a.n - at < 8 ? (int)(a.n - at) : 8;
        const bool whole = VEC && many == 8;
        if (whole) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                in.raw[j] = reinterpret_cast<const uint4 *>(x + at)[j];
                if (RES) add.raw[j] = reinterpret_cast<const uint4 *>(res + at)[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < many) {
                    in.v[j] = x[at + j];
                    if (RES) add.v[j] = res[at + j];
                }
        }
        const Philox r(seed, number, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const W kept = r.half(j) >= a.threshold ? widen<T>(in.v[j]) * factor : (W)0;
            in.v[j] = narrow<T>(RES ? kept + widen<T>(add.v[j]) : kept);
        }
        if (whole) {
#pragma unroll
            for (int j = 0; j < P; ++j) reinterpret_cast<uint4 *>(out + at)[j] = in.raw[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < many) out[at + j] = in.v[j];
        }
    }
}

__global__ void dropout_next_kernel(int64_t *state, int64_t *drawn) {
    drawn[0] = state[0];
    drawn[1] = (int64_t)atomicAdd(reinterpret_cast<unsigned long long *>(state + 1), 1ull);
}

template <typename T> cudaError_t launch(const DropArgs &a, cudaStream_t stream) {
    const int64_t want = ((a.n + 7) / 8 + kThreads - 1) / kThreads, cap = (int64_t)1 << 30;
    const unsigned blocks = (unsigned)(want < cap ? want : cap);
    const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                       reinterpret_cast<uintptr_t>(a.out)) % 16) == 0;
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
    msda::DropArgs a = {x, residual, out, counter, n, 0u, 0.0, nullptr};
    a.threshold = (uint32_t)nearbyint(p * 65536.0);
    a.factor = a.threshold < 65536u ? 65536.0 / (65536.0 - a.threshold) : 0.0;
    if (msda::fault_word_for_launch(&a.err) != cudaSuccess) return MSDA_ERR_CUDA;
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
