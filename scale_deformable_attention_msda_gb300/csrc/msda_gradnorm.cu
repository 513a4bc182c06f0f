// The global norm of a list of gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over all entries of g^2), or max |g|
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// A launch takes a table of up to kLargeTable tensors of one type by value (no
// copy to the device, nothing to keep alive while a graph replays). The tensors
// are cut into units of 4 KB; a warp takes a contiguous run of units, so
// that many small tensors and a few large ones spread over the SMs alike. The
// first kernel leaves one partial result per block; every block of the second
// adds them up in the same order (the norm has the same bits in all of them,
// and from call to call) and scales its units, last to first: those the L2
// still holds from the first kernel come first.
//
// A list of up to kSmallTable tensors and kSmallUnits units takes one launch of a
// single cluster instead, whose blocks exchange their partial results through
// distributed shared memory. A layer's ten tensors take 8.8 us so, 7.0 as two
// launches in a graph, but a call from the host 15 us instead of 20; past a unit a
// warp the cluster's 8 SMs are too few (512 units: 12.6 us).
//
// What bounds it: memory, over two passes of the gradients. 300 million bf16
// entries into fp32 take 386 us (2.4 GB with the second read, 6.2 TB/s); a
// detector's 339 fp32 tensors, 163 MB, into another buffer 83 us (the L2 saves 49
// of the second read's 163 MB), their norm alone 31 us; the largest of 60 million
// fp16 entries 24 us. fp64 arithmetic is kept to a few additions per block: with
// fp64 sums in every lane and a square root and a division in every thread, the
// same calls took 392, 86, 34 and 29 us. (GB300, calls in a graph.)
#include <cooperative_groups.h>
#include <float.h>

#include <type_traits>

#include "msda_common.cuh"
#include "msda_host.h"

namespace msda {
cudaError_t fault_word_for_launch(unsigned **err);

namespace {

constexpr int kUnitBytes = 4096;         // of the source: eight 16-byte loads per lane
constexpr int kNormThreads = 256;
constexpr int kSMs = 152, kMaxPerSM = 16, kMaxBlocks = kSMs * kMaxPerSM;   // of one launch
// tensors of a launch: its parameters, the table among them, may fill 32,764 bytes
constexpr int kSmallTable = 64, kLargeTable = 960;
constexpr int kSmallBlocks = 8, kSmallThreads = 1024, kSmallUnits = 256;
constexpr int64_t kMaxEntries = (int64_t)1 << 38;   // of one tensor: its units fit 2^29

// Tensors of a launch: source, destination, entries, and the units before each.
template <int N> struct Table {
    const void *src[N];
    void *dst[N];
    int64_t size[N];
    uint32_t before[N + 1];
    int count;
    uint16_t start[kMaxBlocks];          // tensor in which a block's first unit lies
};

// First unit of warp w of `warps`: units / warps each, the first units % warps
// one more.
__host__ __device__ inline uint32_t first_unit(uint32_t units, uint32_t warps, uint32_t w) {
    const uint32_t each = units / warps, more = units % warps;
    return w * each + (w < more ? w : more);
}

static_assert(sizeof(Table<kLargeTable>) <= 32764 - 64, "a launch's parameters");

struct Run { uint32_t begin, end; };     // a warp's units

template <int N, int TH = kNormThreads> __device__ __forceinline__ Run warp_run(const Table<N> &t) {
    const uint32_t units = t.before[t.count], warps = gridDim.x * (TH / 32);
    const uint32_t w = blockIdx.x * (TH / 32) + threadIdx.x / 32;
    return Run{first_unit(units, warps, w), first_unit(units, warps, w + 1)};
}

// Index of the tensor that unit u of the block lies in.
template <int N> __device__ __forceinline__ int tensor_of(const Table<N> &t, uint32_t u) {
    int i = t.start[blockIdx.x];
    while (u >= t.before[i + 1]) ++i;
    return i;
}

// A unit's entries [begin, end) of its tensor. The unit boundaries lie on
// 16-byte boundaries of the source; the first unit takes the entries before its
// first boundary as well, [0, body).
template <typename T> struct Unit {
    int64_t begin, end, body;
    __device__ __forceinline__ Unit(const T *src, int64_t size, uint32_t at) {
        constexpr int per = kUnitBytes / sizeof(T);
        const int64_t head = (16 - (reinterpret_cast<uintptr_t>(src) & 15)) % 16 / sizeof(T);
        body = head + (int64_t)at * per;
        begin = at == 0 ? 0 : body;
        end = body + per < size ? body + per : size;
        if (body > end) body = end;
    }
};

// Checked build: entries [at, at + n) lie in a tensor of `size`.
__device__ __forceinline__ bool entries_ok(int64_t at, int64_t n, int64_t size, unsigned *err) {
#ifdef MSDA_CHECKED
    const bool ok = at >= 0 && at <= size - n;
    if (!ok && err) atomicOr(err, 1u);
    return ok;
#else
    return true;
#endif
}

// Checked build: the unit lies in its tensor, and its tensor in the table.
template <typename T>
__device__ __forceinline__ bool unit_ok(const Unit<T> &u, int64_t size, int tensor, int count, unsigned *err) {
#ifdef MSDA_CHECKED
    const bool ok = u.begin >= 0 && u.end <= size && u.begin <= u.end && tensor >= 0 && tensor < count;
    if (!ok && err) atomicOr(err, 1u);
    return ok;
#else
    return true;
#endif
}

template <typename T> __host__ __device__ uint32_t units_of(const void *src, int64_t size) {
    constexpr int64_t per = kUnitBytes / sizeof(T);
    const int64_t head = (16 - (reinterpret_cast<uintptr_t>(src) & 15)) % 16 / sizeof(T);
    const int64_t body = size > head ? size - head : 0;
    return size == 0 ? 0u : body == 0 ? 1u : (uint32_t)((body + per - 1) / per);
}

template <typename T> __device__ __forceinline__ double as_double(T v) {
    if constexpr (sizeof(T) == 8) return v;
    else return (double)Elem<T>::to_f(v);
}

// The larger of two; NaN if either is.
__device__ __forceinline__ double larger(double a, double b) { return a > b || a != a ? a : b; }

template <bool LARGEST> __device__ __forceinline__ double join(double a, double b) {
    return LARGEST ? larger(a, b) : a + b;
}

// A lane's vectors of a unit, zeros where it has none. A whole unit's loads are
// issued together: where each depends on a test of its own the compiler spreads
// them out, and the norm of a detector's gradients takes 37.8 us instead of 30.7.
template <int PER>
__device__ __forceinline__ void load_unit(uint4 (&raw)[PER], const uint4 *from, int vectors, int lane) {
    if (vectors == kUnitBytes / 16) {
#pragma unroll
        for (int k = 0; k < kUnitBytes / 512; ++k) raw[k] = from[k * 32 + lane];
        return;
    }
#pragma unroll
    for (int k = 0; k < kUnitBytes / 512; ++k) {
        raw[k] = make_uint4(0u, 0u, 0u, 0u);
        if (k * 32 + lane < vectors) raw[k] = from[k * 32 + lane];
    }
}

// One lane's share of its warp's units. Of 16- and 32-bit entries the squares are
// added in fp32, 34 or 66 of them, and these sums in a pair of fp32 with the error
// of every addition carried along: fp64 runs at a sixtieth of fp32's rate here.
// Where a unit's sum is not finite, or would leave that range later (1e30), or is
// so small that squares lost digits (under 1e-36: 66 roundings of subnormals,
// 2^-150 each, are 2^-24 of it) though not all entries are zero, the entries are
// squared and added in fp64 instead. The largest entry is kept as the bits of its
// absolute value, which order like the values, NaN above infinity.
struct Share {
    float hi = 0.0f, lo = 0.0f;
    double wide = 0.0;
    uint32_t top = 0u;
    __device__ __forceinline__ void add(float v) {
        const float s = hi + v, b = s - hi;
        lo += (hi - (s - b)) + (v - b);
        hi = s;
    }
};

template <typename T> __device__ __forceinline__ uint32_t abs_bits(T v) {
    return __float_as_uint(Elem<T>::to_f(v)) & 0x7fffffffu;
}

template <typename T, bool LARGEST>
__device__ __forceinline__ void add_unit(Share &share, const T *src, const Unit<T> &u, int lane) {
    constexpr int V = 16 / sizeof(T), per = kUnitBytes / 16 / 32;
    const int vectors = (int)((u.end - u.body) / V);
    uint4 raw[per];
    load_unit(raw, reinterpret_cast<const uint4 *>(src + u.body), vectors, lane);
    // before the first and after the last whole vector: at most V - 1 entries each
    const int64_t head = u.begin + lane, tail = u.body + (int64_t)vectors * V + lane;
    const bool has_head = head < u.body, has_tail = tail < u.end;
    if constexpr (sizeof(T) == 8) {
        double a = has_head ? src[head] : 0.0, b = has_tail ? src[tail] : 0.0;
        share.wide = LARGEST ? larger(larger(share.wide, fabs(a)), fabs(b)) : fma(a, a, fma(b, b, share.wide));
#pragma unroll
        for (int k = 0; k < per; ++k) {
            a = __hiloint2double(raw[k].y, raw[k].x);
            b = __hiloint2double(raw[k].w, raw[k].z);
            share.wide = LARGEST ? larger(larger(share.wide, fabs(a)), fabs(b)) : fma(a, a, fma(b, b, share.wide));
        }
    } else if constexpr (LARGEST) {
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < per; ++k) {
            const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) top = max(top, w[i] & 0x7fffffffu);
                else top = __vmaxu2(top, w[i] & 0x7fff7fffu);
            }
        }
        if constexpr (sizeof(T) == 2) {
            const unsigned short half = (unsigned short)max(top & 0xffffu, top >> 16);
            top = abs_bits(*reinterpret_cast<const T *>(&half));
        }
        if (has_head) top = max(top, abs_bits(src[head]));
        if (has_tail) top = max(top, abs_bits(src[tail]));
        share.top = max(share.top, top);
    } else {
        const float a = has_head ? Elem<T>::to_f(src[head]) : 0.0f, b = has_tail ? Elem<T>::to_f(src[tail]) : 0.0f;
        float sum = fmaf(a, a, b * b);
        uint32_t any = __float_as_uint(a) | __float_as_uint(b);
#pragma unroll
        for (int k = 0; k < per; ++k) {
            float v[V];
            unpack16<T>(v, raw[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(v[i], v[i], sum);
            any |= raw[k].x | raw[k].y | raw[k].z | raw[k].w;
        }
        if (sum >= 1e-36f && sum <= 1e30f) {
            share.add(sum);
        } else if ((any & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) != 0u) {
            double wide = (double)a * a + (double)b * b;
#pragma unroll 1
            for (int k = 0; k < per; ++k) {
                const int at = k * 32 + lane;
                if (at >= vectors) break;
#pragma unroll 1
                for (int i = 0; i < V; ++i) {
                    const double v = as_double<T>(src[u.body + at * V + i]);
                    wide += v * v;
                }
            }
            share.wide += wide;
        }
    }
}

// The shares of a warp's lanes, joined; in lane 0.
template <typename T, bool LARGEST> __device__ __forceinline__ double warp_join(Share share) {
    if constexpr (LARGEST && sizeof(T) != 8) {
        return (double)__uint_as_float(__reduce_max_sync(0xffffffffu, share.top));
    } else {
        if (sizeof(T) != 8 && !__any_sync(0xffffffffu, share.wide != 0.0)) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const float hi = __shfl_xor_sync(0xffffffffu, share.hi, off);
                const float lo = __shfl_xor_sync(0xffffffffu, share.lo, off);
                share.add(hi);
                share.lo += lo;
            }
            return (threadIdx.x & 31) == 0 ? (double)share.hi + (double)share.lo : 0.0;
        }
        double v = sizeof(T) == 8 ? share.wide : share.wide + ((double)share.hi + (double)share.lo);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v = join<LARGEST>(v, __shfl_xor_sync(0xffffffffu, v, off));
        return v;
    }
}

// What a block's warps found (each in its lane 0), joined; in thread 0.
template <bool LARGEST> __device__ __forceinline__ double block_join(double v, double *scratch) {
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < blockDim.x / 32 ? scratch[threadIdx.x] : 0.0;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v = join<LARGEST>(v, __shfl_xor_sync(0xffffffffu, v, off));
    }
    return v;
}

// A warp's units, joined; in lane 0.
template <typename T, bool LARGEST, int N>
__device__ __forceinline__ double run_part(const Table<N> &t, const Run &run, unsigned *err) {
    const int lane = threadIdx.x & 31;
    Share share;
    if (run.begin < run.end) {
        int i = tensor_of(t, run.begin);
        for (uint32_t u = run.begin; u < run.end; ++u) {
            while (u >= t.before[i + 1]) ++i;
            const T *src = static_cast<const T *>(t.src[i]);
            const Unit<T> unit(src, t.size[i], u - t.before[i]);
            if (!unit_ok(unit, t.size[i], i, t.count, err)) continue;
            add_unit<T, LARGEST>(share, src, unit, lane);
        }
    }
    return warp_join<T, LARGEST>(share);
}

template <typename T, bool LARGEST, int N>
__global__ void __launch_bounds__(kNormThreads)
grad_part_kernel(const __grid_constant__ Table<N> t, double *partial, unsigned *err) {
    __shared__ double scratch[32];
    cudaTriggerProgrammaticLaunchCompletion();
    const double part = block_join<LARGEST>(run_part<T, LARGEST>(t, warp_run(t), err), scratch);
    if (threadIdx.x == 0) partial[blockIdx.x] = part;
}

// The partial results of all blocks, joined in a fixed order; in the first warp.
// All threads read, so that the reads wait for each other little, and few add:
// fp64 is what every block's start waits for.
template <bool LARGEST>
__device__ __forceinline__ double join_all(const double *partial, int count, double (&scratch)[kNormThreads]) {
    double v = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < count; i += kNormThreads) v = join<LARGEST>(v, partial[i]);
    scratch[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        double a = v, b = scratch[threadIdx.x + kNormThreads / 2];
#pragma unroll
        for (int i = 32; i < kNormThreads / 2; i += 32) {
            a = join<LARGEST>(a, scratch[threadIdx.x + i]);
            b = join<LARGEST>(b, scratch[threadIdx.x + kNormThreads / 2 + i]);
        }
        v = join<LARGEST>(a, b);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v = join<LARGEST>(v, __shfl_xor_sync(0xffffffffu, v, off));
    }
    return v;
}

// The norm from what all blocks found (`total`), by one thread.
template <bool LARGEST> __device__ __forceinline__ double norm_of(double total) {
    return LARGEST ? total : sqrt(total);
}

__device__ __forceinline__ void write_norm(double norm, void *to, bool wide) {
    if (wide) *static_cast<double *>(to) = norm;
    else *static_cast<float *>(to) = (float)norm;
}

template <bool LARGEST>
__global__ void __launch_bounds__(kNormThreads)
grad_norm_kernel(const double *partial, int count, void *norm, bool wide) {
    __shared__ double scratch[kNormThreads];
    cudaGridDependencySynchronize();
    const double total = join_all<LARGEST>(partial, count, scratch);
    if (threadIdx.x == 0) write_norm(norm_of<LARGEST>(total), norm, wide);
}

// 32 bytes in one store (the address a multiple of 32).
__device__ __forceinline__ void store32(float *to, const float *v) {
    asm volatile("st.global.cs.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// The 16 bytes that start `bytes` (under 16, a multiple of 2) into a lane's
// vector and run into the next lane's; lane 31 is followed by lane 0's `next`.
__device__ __forceinline__ void shift_in(uint4 &own, const uint4 &next, int lane, int bytes) {
    const uint4 give = lane == 0 ? next : own;
    uint32_t w[8] = {own.x, own.y, own.z, own.w};
    const uint32_t g[4] = {give.x, give.y, give.z, give.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 + i] = __shfl_sync(0xffffffffu, g[i], (lane + 1) & 31);
    if (bytes & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (bytes & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    own = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T> __device__ __forceinline__ void put(T *to, float v) { *to = Elem<T>::from_f(v); }
__device__ __forceinline__ void put(double *to, double v) { *to = v; }

// min(1, max_norm / (norm + 1e-6)) as value * again; NaN stays NaN. `again` is 1 but
// for factors below the type's normal numbers, which would have lost digits: those
// are kept larger by a power of two and entries multiplied by its inverse after.
template <typename T> using Arith = typename std::conditional<sizeof(T) == 8, double, float>::type;
template <typename T> struct Factor {
    Arith<T> value, again;
    __device__ __forceinline__ Arith<T> operator()(Arith<T> v) const { return v * value * again; }
};
template <typename T> __device__ __forceinline__ Factor<T> factor_of(double max_norm, double norm) {
    using A = Arith<T>;
    constexpr double least = sizeof(A) == 8 ? DBL_MIN : (double)FLT_MIN;   // 2^-1022, 2^-126
    const double ratio = max_norm / (norm + 1e-6);
    if (!(ratio < least)) return {(A)(ratio > 1.0 ? 1.0 : ratio), (A)1};
    // of doubles the quotient itself lost digits
    if constexpr (sizeof(A) == 8) return {max_norm / least / (norm + 1e-6), least};
    else return {(A)(ratio / least), (A)least};
}

// A warp's units, last to first, times the factor.
template <typename T, typename U, int N>
__device__ __forceinline__ void run_scale(const Table<N> &t, const Run &run, Factor<T> factor, unsigned *err) {
    using A = Arith<T>;
    constexpr int V = 16 / sizeof(T), per = kUnitBytes / 16 / 32;
    if (run.begin >= run.end) return;
    const int lane = threadIdx.x & 31;
    int i = tensor_of(t, run.end - 1);
#pragma unroll 1
    for (uint32_t u = run.end; u-- > run.begin;) {
        while (u < t.before[i]) --i;
        const T *src = static_cast<const T *>(t.src[i]);
        U *dst = static_cast<U *>(t.dst[i]);
        if (factor.value == (A)1 && factor.again == (A)1 &&
            static_cast<const void *>(src) == static_cast<const void *>(dst)) continue;
        const Unit<T> unit(src, t.size[i], u - t.before[i]);
        if (!unit_ok(unit, t.size[i], i, t.count, err)) continue;
        // A source vector's entries go out in one store of 16 or 32 bytes. Where the
        // destination's boundaries lie `skew` entries after the source's, a store
        // takes entries of two source vectors, a lane's own and the next lane's.
        constexpr int out = V * sizeof(U);
        const int skew = (int)((out - (reinterpret_cast<uintptr_t>(dst + unit.body) & (out - 1))) % out / sizeof(U));
        const int vectors = (int)((unit.end - unit.body) / V);
        const int whole = skew ? (vectors ? vectors - 1 : 0) : vectors;      // stores
        const int64_t from = whole ? unit.body + skew : unit.body, to = from + (int64_t)whole * V;
        uint4 raw[per + 1];
#pragma unroll
        for (int k = 0; k < per; ++k) {
            const int at = k * 32 + lane;
            raw[k] = make_uint4(0u, 0u, 0u, 0u);
            if (at < vectors && entries_ok(unit.body + at * V, V, t.size[i], err)) raw[k] = __ldcs(reinterpret_cast<const uint4 *>(src + unit.body + at * V));
        }
        raw[per] = make_uint4(0u, 0u, 0u, 0u);
        for (int64_t j = unit.begin + lane; j < from; j += 32)
            if (entries_ok(j, 1, t.size[i], err)) put(dst + j, factor((A)as_double<T>(src[j])));
        for (int64_t j = to + lane; j < unit.end; j += 32)
            if (entries_ok(j, 1, t.size[i], err)) put(dst + j, factor((A)as_double<T>(src[j])));
#pragma unroll
        for (int k = 0; k < per; ++k) {
            if (skew) shift_in(raw[k], raw[k + 1], lane, skew * (int)sizeof(T));
            const int at = k * 32 + lane;
            if (at >= whole || !entries_ok(from + at * V, V, t.size[i], err)) continue;
            U *where = dst + from + at * V;
            if constexpr (sizeof(T) == 8) {
                __stcs(reinterpret_cast<double2 *>(where),
                       make_double2(factor(__hiloint2double(raw[k].y, raw[k].x)),
                                    factor(__hiloint2double(raw[k].w, raw[k].z))));
            } else {
                float v[V];
                unpack16<T>(v, raw[k]);
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] *= factor.value;
                if (factor.again != 1.0f) {      // (multiplied always, a detector's list takes 84.1 us, not 82.8)
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] *= factor.again;
                }
                if constexpr (out == 32) store32(where, v);
                else __stcs(reinterpret_cast<uint4 *>(where), pack16<U>(v));
            }
        }
    }
}

template <typename T, typename U, bool LARGEST, int N>
__global__ void __launch_bounds__(kNormThreads)
grad_scale_kernel(const __grid_constant__ Table<N> t, const double *partial, int count, double max_norm,
                  void *norm, bool wide, unsigned *err) {
    __shared__ double scratch[kNormThreads];
    __shared__ Factor<T> factor;
    cudaGridDependencySynchronize();
    const double total = join_all<LARGEST>(partial, count, scratch);
    if (threadIdx.x == 0) {
        const double n = norm_of<LARGEST>(total);
        if (norm && blockIdx.x == 0) write_norm(n, norm, wide);
        factor = factor_of<T>(max_norm, n);
    }
    __syncthreads();
    run_scale<T, U>(t, warp_run(t), factor, err);
}

// The whole of a small list in one cluster: the blocks' partial results are read
// through distributed shared memory, in the same order by all.
template <typename T, typename U, bool LARGEST>
__global__ void __cluster_dims__(kSmallBlocks, 1, 1) __launch_bounds__(kSmallThreads)
grad_small_kernel(const __grid_constant__ Table<kSmallTable> t, bool scale, double max_norm, void *norm, bool wide,
                  unsigned *err) {
    __shared__ double scratch[32], mine;
    __shared__ Factor<T> factor;
    const auto cluster = cooperative_groups::this_cluster();
    const Run run = warp_run<kSmallTable, kSmallThreads>(t);
    const double part = block_join<LARGEST>(run_part<T, LARGEST>(t, run, err), scratch);
    if (threadIdx.x == 0) mine = part;
    cluster.sync();
    if (threadIdx.x == 0) {
        double total = 0.0;
        for (int b = 0; b < kSmallBlocks; ++b) total = join<LARGEST>(total, *cluster.map_shared_rank(&mine, b));
        const double n = norm_of<LARGEST>(total);
        if (blockIdx.x == 0) write_norm(n, norm, wide);
        factor = factor_of<T>(max_norm, n);
    }
    cluster.sync();                      // no block leaves while another reads its part
    if (scale) run_scale<T, U>(t, run, factor, err);
}

// ----------------------------------------------------------------- launches

int bytes_of(int32_t dt) { return dt == MSDA_F64 ? 8 : dt == MSDA_F32 ? 4 : 2; }

// Tensors of a list that share a launch: one type of source and destination.
bool in_class(const msda_grad_list_t &l, int64_t i, int32_t from, int32_t to) {
    return l.sizes[i] > 0 && l.dtypes[i] == from && (to < 0 || l.out_dtypes[i] == to);
}

uint32_t units_for(int32_t dt, const void *src, int64_t size) {
    switch (dt) {
        case MSDA_F64: return units_of<double>(src, size);
        case MSDA_F32: return units_of<float>(src, size);
        case MSDA_BF16: return units_of<__nv_bfloat16>(src, size);
        default: return units_of<__half>(src, size);
    }
}

// Blocks of a launch over `units`: a warp per unit up to two blocks an SM; then
// so many that a warp has about seven units, 3 to 16 blocks an SM, and of two
// neighbouring counts the one that leaves the last round of units fuller.
// Measured at 3, 5, 8, 12 and 16 blocks an SM: the norm of 60 million fp16
// entries (29,000 units) takes 27.4, 28.5, 32.3, 35.9 and 39.6 us, clipping 300
// million bf16 into fp32 (146,000 units) 437, 413, 409, 400 and 388 us: few
// units a warp spend their time on the partial results, many end unevenly.
int blocks_for(uint32_t units) {
    const uint32_t warps = kNormThreads / 32;
    if (units <= 2 * kSMs * warps) return (int)((units + warps - 1) / warps);
    uint32_t least = units / (kSMs * warps * 7);
    least = least < 3 ? 3 : least > kMaxPerSM - 1 ? kMaxPerSM - 1 : least;
    const uint32_t most = least == 3 ? 6 : least + 1;
    int best = 0;
    uint64_t waste = ~0ull;
    for (uint32_t per_sm = least; per_sm <= most; ++per_sm) {
        const uint64_t all = (uint64_t)per_sm * kSMs * warps, left = (units + all - 1) / all * all - units;
        if (left < waste) {
            waste = left;
            best = (int)(per_sm * kSMs);
        }
    }
    return best;
}

cudaError_t launch(const void *kernel, int blocks, void **args, bool early, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <typename T, int N> const void *part_kernel(bool largest) {
    return largest ? (const void *)grad_part_kernel<T, true, N> : (const void *)grad_part_kernel<T, false, N>;
}
template <typename T, typename U, int N> const void *scale_kernel(bool largest) {
    return largest ? (const void *)grad_scale_kernel<T, U, true, N> : (const void *)grad_scale_kernel<T, U, false, N>;
}
template <int N> const void *part_kernel(int32_t dt, bool largest) {
    switch (dt) {
        case MSDA_F64: return part_kernel<double, N>(largest);
        case MSDA_F32: return part_kernel<float, N>(largest);
        case MSDA_BF16: return part_kernel<__nv_bfloat16, N>(largest);
        default: return part_kernel<__half, N>(largest);
    }
}
template <int N> const void *scale_kernel(int32_t dt, int32_t to, bool largest) {
    if (dt == MSDA_F64) return scale_kernel<double, double, N>(largest);
    if (dt == MSDA_F32) return scale_kernel<float, float, N>(largest);
    if (dt == MSDA_BF16)
        return to == MSDA_F32 ? scale_kernel<__nv_bfloat16, float, N>(largest)
                              : scale_kernel<__nv_bfloat16, __nv_bfloat16, N>(largest);
    return to == MSDA_F32 ? scale_kernel<__half, float, N>(largest) : scale_kernel<__half, __half, N>(largest);
}

// Adds the tensors of one class to a table, in the list's order from tensor i,
// until it is full; returns the tensor to go on from.
template <int N>
int64_t fill(const msda_grad_list_t &l, int32_t from, int32_t to, int64_t i, Table<N> *t) {
    t->count = 0;
    t->before[0] = 0;
    for (; i < l.count; ++i) {
        if (!in_class(l, i, from, to)) continue;
        const uint32_t units = units_for(from, l.grads[i], l.sizes[i]);
        if (t->count == N || units > 0x7fffffffu - t->before[t->count]) break;
        t->src[t->count] = l.grads[i];
        t->dst[t->count] = to < 0 ? nullptr : l.outs[i];
        t->size[t->count] = l.sizes[i];
        t->before[t->count + 1] = t->before[t->count] + units;
        ++t->count;
    }
    return i;
}

// The tensors in which the first units of the blocks, of `per` warps, lie.
template <int N> void set_starts(Table<N> &t, int blocks, uint32_t per) {
    const uint32_t units = t.before[t.count];
    int i = 0;
    for (int b = 0; b < blocks; ++b) {
        const uint32_t u = first_unit(units, blocks * per, b * per);
        while (i + 1 < t.count && u >= t.before[i + 1]) ++i;
        t.start[b] = (uint16_t)i;
    }
}

// Hands the tensors of one class to `run(table, blocks)`, a table at a time.
// Stops at the first error.
template <int N, typename F>
cudaError_t each_table(const msda_grad_list_t &l, int32_t from, int32_t to, F run) {
    Table<N> t;
    for (int64_t i = 0; i < l.count;) {
        i = fill<N>(l, from, to, i, &t);
        if (!t.count) break;
        const int blocks = blocks_for(t.before[t.count]);
        set_starts(t, blocks, kNormThreads / 32);
        const cudaError_t e = run(t, blocks);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// What one pass over a list finds: per type (msda_dtype_t's values), whether it
// occurs, with a destination of its own type or fp32, and the launches the first
// kernel may need.
constexpr int kTypes = 4;
struct Summary {
    int64_t count[kTypes], units[kTypes];
    bool to_own[kTypes], to_f32[kTypes];
    bool f64;
    // a table per kLargeTable tensors, and one more each time that units fill one
    int64_t launches() const {
        int64_t n = 0;
        for (int dt = 0; dt < kTypes; ++dt)
            if (count[dt]) n += (count[dt] + kLargeTable - 1) / kLargeTable + (units[dt] >> 30);
        return n;
    }
    size_t bytes() const {
        const int64_t n = launches();
        return (size_t)(n < 1 ? 1 : n) * kMaxBlocks * sizeof(double);
    }
};

msda_status_t check(const msda_grad_list_t *l, bool clip, int kind, Summary *s) {
    *s = Summary{};
    if (!l) return MSDA_ERR_NULL;
    if (l->count < 0 || l->count > (1 << 24)) return MSDA_ERR_SHAPE;
    if (kind != MSDA_NORM_2 && kind != MSDA_NORM_INF) return MSDA_ERR_DTYPE;
    if (l->count == 0) return MSDA_OK;
    if (!l->grads || !l->sizes || !l->dtypes || (clip && (!l->outs || !l->out_dtypes))) return MSDA_ERR_NULL;
    for (int64_t i = 0; i < l->count; ++i) {
        if (l->sizes[i] < 0 || l->sizes[i] > kMaxEntries) return MSDA_ERR_SHAPE;
        const int32_t dt = l->dtypes[i];
        if (dt < 0 || dt >= kTypes) return MSDA_ERR_DTYPE;
        s->f64 = s->f64 || dt == MSDA_F64;
        if (clip) {
            const int32_t to = l->out_dtypes[i];
            if (to != dt && !(to == MSDA_F32 && bytes_of(dt) == 2)) return MSDA_ERR_DTYPE;
            (to == dt ? s->to_own : s->to_f32)[dt] = true;
        }
        if (l->sizes[i] == 0) continue;
        if (!l->grads[i] || (clip && !l->outs[i])) return MSDA_ERR_NULL;
        if (reinterpret_cast<uintptr_t>(l->grads[i]) % bytes_of(dt)) return MSDA_ERR_ALIGN;
        if (clip && reinterpret_cast<uintptr_t>(l->outs[i]) % bytes_of(l->out_dtypes[i])) return MSDA_ERR_ALIGN;
        ++s->count[dt];
        s->units[dt] += units_for(dt, l->grads[i], l->sizes[i]);
    }
    return MSDA_OK;
}

// First kernel over the whole list; *parts: partial results written.
template <int N>
cudaError_t launch_parts(const msda_grad_list_t &l, const Summary &sum, bool largest, double *partial, int *parts,
                         unsigned *err, cudaStream_t stream) {
    *parts = 0;
    for (int32_t dt = 0; dt < kTypes; ++dt) {
        if (!sum.count[dt]) continue;
        const cudaError_t e = each_table<N>(l, dt, -1, [&](Table<N> &t, int blocks) {
            double *to = partial + *parts;
            void *args[] = {&t, &to, &err};
            *parts += blocks;
            return launch(part_kernel<N>(dt, largest), blocks, args, false, stream);
        });
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int N>
cudaError_t launch_scale(const msda_grad_list_t &l, const Summary &sum, bool largest, const double *partial,
                         int parts, double max_norm, void *norm, unsigned *err, cudaStream_t stream) {
    bool first = true, wide = sum.f64;
    for (int32_t dt = 0; dt < kTypes; ++dt) {
        for (int own = 0; own < 2; ++own) {
            if (!sum.count[dt] || !(own ? sum.to_own : sum.to_f32)[dt]) continue;
            const int32_t to = own ? dt : (int32_t)MSDA_F32;
            const cudaError_t e = each_table<N>(l, dt, to, [&](Table<N> &t, int blocks) {
                void *where = first ? norm : nullptr;
                void *args[] = {&t, &partial, &parts, &max_norm, &where, &wide, &err};
                const bool early = first;        // only this one follows the first kernel directly
                first = false;
                return launch(scale_kernel<N>(dt, to, largest), blocks, args, early, stream);
            });
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

template <typename T, typename U> const void *small_kernel(bool largest) {
    return largest ? (const void *)grad_small_kernel<T, U, true> : (const void *)grad_small_kernel<T, U, false>;
}
const void *small_kernel(int32_t dt, int32_t to, bool largest) {
    if (dt == MSDA_F64) return small_kernel<double, double>(largest);
    if (dt == MSDA_F32) return small_kernel<float, float>(largest);
    if (dt == MSDA_BF16)
        return to == MSDA_F32 ? small_kernel<__nv_bfloat16, float>(largest)
                              : small_kernel<__nv_bfloat16, __nv_bfloat16>(largest);
    return to == MSDA_F32 ? small_kernel<__half, float>(largest) : small_kernel<__half, __half>(largest);
}

// Whether one cluster takes the list: its tensors fit the small table, are of one
// type of source and destination, and few units.
bool is_small(const msda_grad_list_t &l, const Summary &sum, bool clip, int32_t *from, int32_t *to) {
    int classes = 0;
    for (int32_t dt = 0; dt < kTypes; ++dt) {
        if (!sum.count[dt]) continue;
        if (sum.units[dt] > kSmallUnits || (clip && sum.to_own[dt] && sum.to_f32[dt])) return false;
        ++classes;
        *from = dt;
        *to = clip && sum.to_f32[dt] ? (int32_t)MSDA_F32 : dt;
    }
    return l.count <= kSmallTable && classes == 1;
}

cudaError_t launch_small(const msda_grad_list_t &l, const Summary &sum, bool largest, bool clip, double max_norm,
                         void *norm, int32_t from, int32_t to, cudaStream_t stream) {
    unsigned *err = nullptr;
    const cudaError_t e = fault_word_for_launch(&err);
    if (e != cudaSuccess) return e;
    Table<kSmallTable> t;
    fill<kSmallTable>(l, from, clip ? to : -1, 0, &t);
    set_starts(t, kSmallBlocks, kSmallThreads / 32);
    bool wide = sum.f64;
    void *args[] = {&t, &clip, &max_norm, &norm, &wide, &err};
    return cudaLaunchKernel(small_kernel(from, to, largest), dim3(kSmallBlocks), dim3(kSmallThreads), args, 0, stream);
}

cudaError_t launch_norm(bool largest, const double *partial, int parts, void *norm, bool wide, cudaStream_t stream) {
    void *args[] = {&partial, &parts, &norm, &wide};
    return launch(largest ? (const void *)grad_norm_kernel<true> : (const void *)grad_norm_kernel<false>, 1, args,
                  true, stream);
}

template <int N>
cudaError_t norm_and_scale(const msda_grad_list_t &l, const Summary &sum, bool largest, bool clip, double max_norm,
                           void *norm, double *partial, cudaStream_t stream) {
    unsigned *err = nullptr;
    cudaError_t e = fault_word_for_launch(&err);
    int parts = 0;
    if (e == cudaSuccess) e = launch_parts<N>(l, sum, largest, partial, &parts, err, stream);
    if (e != cudaSuccess) return e;
    if (!clip || parts == 0) return launch_norm(largest, partial, parts, norm, sum.f64, stream);
    return launch_scale<N>(l, sum, largest, partial, parts, max_norm, norm, err, stream);
}

msda_status_t run(const msda_grad_list_t *l, int kind, bool clip, double max_norm, void *norm, void *workspace,
                  size_t workspace_bytes, void *stream) {
    Summary sum;
    const msda_status_t st = check(l, clip, kind, &sum);
    if (st != MSDA_OK) return st;
    if (clip && !(max_norm >= 0.0)) return MSDA_ERR_SHAPE;
    if (!norm) return MSDA_ERR_NULL;
    if (!workspace || workspace_bytes < sum.bytes()) return MSDA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return MSDA_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(norm) % (sum.f64 ? 8 : 4)) return MSDA_ERR_ALIGN;
    double *partial = static_cast<double *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool largest = kind == MSDA_NORM_INF;
    int32_t from, to;
    if (is_small(*l, sum, clip, &from, &to))
        return launch_small(*l, sum, largest, clip, max_norm, norm, from, to, s) == cudaSuccess ? MSDA_OK
                                                                                               : MSDA_ERR_CUDA;
    const cudaError_t e = l->count <= kSmallTable
                              ? norm_and_scale<kSmallTable>(*l, sum, largest, clip, max_norm, norm, partial, s)
                              : norm_and_scale<kLargeTable>(*l, sum, largest, clip, max_norm, norm, partial, s);
    return e == cudaSuccess ? MSDA_OK : MSDA_ERR_CUDA;
}

}  // namespace
}  // namespace msda

extern "C" {

size_t msda_grad_norm_workspace_bytes(const msda_grad_list_t *list) {
    msda::Summary sum;
    return msda::check(list, false, MSDA_NORM_2, &sum) == MSDA_OK ? sum.bytes() : 0;
}

msda_status_t msda_grad_norm(const msda_grad_list_t *list, int kind, void *norm, void *workspace,
                             size_t workspace_bytes, void *stream) {
    return msda::run(list, kind, false, 0.0, norm, workspace, workspace_bytes, stream);
}

msda_status_t msda_clip_grad_norm(const msda_grad_list_t *list, int kind, double max_norm, void *norm,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    return msda::run(list, kind, true, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
