// Attention of 16-bit data on the tensor cores.
//
// A block holds 128 rows (queries, or keys in kGradKV) and walks tiles of BN
// columns, in the three modes of msda_attention.cuh:
//
//            scores                  second product
// kForward   S = Q K'                O += P V
// kGradQ     S = Q K', dP = dO V'    dQ += dS K
// kGradKV    S = K Q', dP = V dO'    dV += P dO, dK += dS Q
//
// One warp fetches tiles with TMA, one issues the scores' MMAs, one those of the
// second products, and in kGradKV one makes an operand of the queries' statistics
// (tc_bias_row). The other warps, in groups of four, work on rows: each thread has
// one row of the scores (PARTS 1), or a half of one (PARTS 2), which it reads from
// tensor memory, so that a row's maximum and sum need no exchange between threads.
// The weights go back to tensor memory in 16 bits, as the left operand of the second
// product; nothing of the scores touches shared memory. The same tile in shared
// memory serves as the right operand of both products, read along its rows for the
// scores and across them for the second product.
//
// Roundings: the weights (P, dS) to the data's 16 bits, off by 2^-8 of the value at most in
// bf16 and by 2^-11 in fp16, as the second product's operands have
// to be; all sums, maxima and statistics are fp32.
//
// What bounds it: chains of waits between products, exponentials and conversions; no pipe is
// full. Of 4096 x 4096 scores of 32 heads, bf16, D 32 / 64 / 128:
//   forward     169 / 173 / 239 us, 406 / 793 / 1,150 TFLOP/s; 2^29 exponentials at 16 a
//               clock and SM take 115 us alone (D 64: 63% of their pipe, 34% of the products')
//   backward    458 / 501 / 793 us for 5 products' worth, 375 / 686 / 866 TFLOP/s (it
//               computes 7; D 64: 47% of the exponentials' pipe, 45% of the products')
// Tiles, by what was measured at D 64 unless said otherwise:
//   forward     two blocks of an SM (one waits for its products while the other takes
//               exponentials) of 128 columns. 64 or 96 columns: slower, or the registers
//               spill. D 128: tensor memory leaves 64 columns, and two buffers of weights.
//   backward    one block with two groups of row warps, a half of each row's columns each:
//               531 us when four groups took 578, and three that take tiles in turn were slower
//               than two. D 128 in kGradKV: the weights lie over the scores, so P is released,
//               and its product issued, before dP is waited for.
//   kGradKV for few queries: see tc_short.
#pragma once

#include <cudaTypedefs.h>

#include "msda_attention_host.h"
#include "msda_host.h"
#include "msda_tcgen05.cuh"

namespace msda {

constexpr int kTcRows = 128;

// DP: channels in shared memory. BN: columns of a tile. PARTS: groups of four warps that
// share each row, a part of the columns each. STAGES, EARLY: tiles in shared memory of the
// two column operands. BLOCKS: of an SM, by tensor memory (512 columns) and shared memory.
// WEIGHTS: buffers of weights in tensor memory; 0: they lie in the scores' columns, and the
// next scores wait for the second product.
template <int BN_, int PARTS_, int STAGES_, int EARLY_, int BLOCKS_, int WEIGHTS_> struct TcSizes {
    static constexpr int BN = BN_, PARTS = PARTS_, STAGES = STAGES_, EARLY = EARLY_, BLOCKS = BLOCKS_, WEIGHTS = WEIGHTS_;
};
template <int MODE, int DP, bool SHORT> struct TcConfig;
template <> struct TcConfig<kForward, 32, false> : TcSizes<128, 1, 3, 3, 2, 1> {};
template <> struct TcConfig<kForward, 64, false> : TcSizes<128, 1, 2, 2, 2, 1> {};
template <> struct TcConfig<kForward, 128, false> : TcSizes<64, 1, 2, 2, 2, 2> {};
template <> struct TcConfig<kGradQ, 32, false> : TcSizes<128, 2, 4, 4, 1, 2> {};
template <> struct TcConfig<kGradQ, 64, false> : TcSizes<128, 2, 3, 3, 1, 2> {};
template <> struct TcConfig<kGradQ, 128, false> : TcSizes<128, 2, 2, 2, 1, 2> {};
template <> struct TcConfig<kGradKV, 32, false> : TcSizes<128, 2, 4, 4, 1, 1> {};
template <> struct TcConfig<kGradKV, 64, false> : TcSizes<128, 2, 3, 3, 1, 1> {};
template <> struct TcConfig<kGradKV, 32, true> : TcSizes<64, 1, 2, 2, 2, 1> {};
template <> struct TcConfig<kGradKV, 64, true> : TcSizes<64, 1, 2, 2, 2, 0> {};
template <> struct TcConfig<kGradKV, 128, false> : TcSizes<128, 2, 2, 2, 1, 0> {};

template <int MODE, int DP, bool SHORT> struct Tc : TcConfig<MODE, DP, SHORT> {
    using C = TcConfig<MODE, DP, SHORT>;
    static constexpr int BN = C::BN, PARTS = C::PARTS, STAGES = C::STAGES, EARLY = C::EARLY, WEIGHTS = C::WEIGHTS;
    // SPLIT: P is released, and its product issued, before dP is waited for
    static constexpr bool ALIAS = WEIGHTS == 0, BACK = MODE != kForward, SPLIT = MODE == kGradKV && ALIAS;
    static constexpr int PITCH = DP == 32 ? 64 : 128, PANELS = DP == 128 ? 2 : 1, PANEL = DP == 128 ? 64 : DP;
    static constexpr int ROW_BYTES = kTcRows * PITCH * PANELS, COL_BYTES = BN * PITCH * PANELS;
    static constexpr int ROW_THREADS = PARTS * 128, THREADS = ROW_THREADS + 128, PART = BN / PARTS;
    // registers: 65,536 of an SM, spread evenly at the start and then by need: a row's thread
    // has its scores of a tile in registers, 128 or (PARTS 2) 64 and as many of dP
    static constexpr int REGS_ROW = 208, REGS_OTHER = PARTS == 1 ? 48 : 88;
    static_assert((PARTS * REGS_ROW + REGS_OTHER) * 128 <= 65536 / C::BLOCKS / THREADS / 8 * 8 * THREADS, "registers");
    // tensor memory: scores (and dP), weights, accumulators
    static constexpr int SCORES = BN * (BACK ? 2 : 1), WIDE = BN / 2 * (MODE == kGradKV ? 2 : 1);
    static constexpr int ACC = SCORES + WEIGHTS * WIDE, RESULTS = MODE == kGradKV ? 2 : 1;
    static constexpr int USED = ACC + RESULTS * DP, COLS = USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
    static_assert(BN == tc_columns(MODE, DP, SHORT) && C::BLOCKS == tc_blocks(MODE, DP, SHORT), "what the host plans with");
    static_assert(MODE != kForward || PARTS == 1, "one maximum and sum a row");
    static_assert(USED <= 512 && COLS * C::BLOCKS <= 512, "tensor memory");
    static constexpr int TILES = (BACK ? 2 : 1) * ROW_BYTES + (STAGES + EARLY) * COL_BYTES;
    // of a column tile: the queries' statistics, and the same as an operand (see tc_bias_row)
    static constexpr int STAT_BYTES = MODE == kGradKV ? 8 * BN : 0, BIAS_BYTES = MODE == kGradKV ? 48 * BN : 0;
    static constexpr int ONES_BYTES = MODE == kGradKV ? 48 * kTcRows : 0;
    static constexpr int INFO = 8;
    static_assert(STAGES + 1 <= INFO, "announcements are read before they are written over");
    static constexpr int NEEDED = 1024 + TILES + STAGES * (STAT_BYTES + BIAS_BYTES) + ONES_BYTES + 1024;
    // as much as keeps one block more off the SM, which would only wait for its tensor memory
    static constexpr int LIMIT = 228 * 1024 / (C::BLOCKS + 1);
    static constexpr int SHARED = NEEDED > LIMIT ? NEEDED : LIMIT;
    static_assert(SHARED <= 227 * 1024 && (SHARED + 1024) * C::BLOCKS <= 228 * 1024, "shared memory");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// What a row's weights are relative to, in the exponent's units. NaN where a maximum that is
// finite overflows by the scale: infinity would make every weight 0, as of a query without keys.
__device__ __forceinline__ float tc_reference(float top, float c, float up) {
    const float ref = top == -INFINITY ? -up : fmaf(top, c, -up);
    return ref == INFINITY ? __int_as_float(0x7fffffff) : ref;
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// ds is at most 2 |dO_i| |v_j| p: for fp16 it is scaled by the power of two r that takes
// the largest of these bounds to 2 at most, and so, with p's 2^14, below 2^15 + 2^-10. The
// largest v_j is that of the batch entry's and key head's keys that some query attends. The
// sums of a query's gradient have its dO_i in common; those of the keys' take the largest of
// the head's queries that attend a key.
template <typename T> struct TcScale { static constexpr float forward = 0.0f, backward = 0.0f; };
template <> struct TcScale<__half> { static constexpr float forward = kHalfWeightUp, backward = kHalfUp; };

__device__ __forceinline__ float tc_most(const float *part, int n) {
    float v = 0.0f;
    for (int i = threadIdx.x & 31; i < n; i += 32) v = fmaxf(v, part[i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}
// square: |dO|^2 of the query, kGradQ.
template <int MODE> __device__ __forceinline__ float tc_ds_scale(const AttnArgs &a, const AttnRows &w, float square) {
    const int64_t at = ((int64_t)w.b * a.N + (MODE == kGradKV ? w.head : w.head / a.G)) * a.norms;
    if (MODE == kGradKV) square = tc_most(a.norm_do + at, a.norms);
    const float bound = 2.01f * sqrtf(square) * sqrtf(tc_most(a.norm_v + at, a.norms));
    if (bound == 0.0f || !isfinite(bound)) return 1.0f;
    int e;
    frexpf(bound, &e);                 // bound < 2^e
    return ldexpf(1.0f, min(1 - e, 100));
}
template <typename T> __device__ __forceinline__ float tc_square(const T *row, int D) {
    float square = 0.0f;
    for (int d = 0; d < D; d += 8) {
        float x[8];
        unpack16<T>(x, ldg16(row + d));
#pragma unroll
        for (int k = 0; k < 8; ++k) square = fmaf(x[k], x[k], square);
    }
    return square;
}

// 32 channels of a row: of the output, or of this split's part (scaled by g), and of
// the output's rounding error.
template <typename T, int MODE>
__device__ __forceinline__ void tc_store(const AttnArgs &a, int64_t row, int split, int which, int d0, const float *v,
                                         float f, float g) {
    if (!attn_ok(a, row, a.part_rows)) return;
    if (a.splits > 1) {
        float *to = a.part + ((int64_t)(which * a.splits + split) * a.part_rows + row) * a.D;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            if (d0 + i < a.D)
                *reinterpret_cast<float4 *>(to + d0 + i) = make_float4(v[i] * g, v[i + 1] * g, v[i + 2] * g, v[i + 3] * g);
        return;
    }
    T *to = static_cast<T *>(MODE == kForward ? a.out : MODE == kGradQ ? a.gq : which ? a.gk : a.gv) + row * a.D;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        if (d0 + i >= a.D) break;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = v[i + k] * f;
        const uint4 packed = pack16<T>(x);
        *reinterpret_cast<uint4 *>(to + d0 + i) = packed;
        if (MODE == kForward && a.rest) {
            float y[8];
            unpack16<T>(y, packed);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] -= y[k];
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.rest) + row * a.D + d0 + i) = pack16<T>(x);
        }
    }
}

// What the fetching lane tells the others of a column tile; cls 0: there is none more.
struct TcTile {
    int pos, head, cls;
};

// Barriers of a buffer of weights: column tile `it` is ready for its second product, or
// done with it. Each buffer has its own: a wait tells a phase only from the one before
// it, and a warp may be ready with the next tile before another is with this one.
template <int WEIGHTS> __device__ __forceinline__ uint64_t *tc_bar(uint64_t *bars, int it) {
    return bars + (WEIGHTS == 2 ? it & 1 : 0);
}
template <int WEIGHTS> __device__ __forceinline__ uint32_t tc_phase(int it) { return (WEIGHTS == 2 ? it >> 1 : it) & 1; }

// kGradKV: -lse and -delta of the columns' queries, added to the scores and to dP by one
// more step of their products: 1, 1, 1 times the three parts that a number has in bf16,
// which together hold its fp32 digits. Read from shared memory by the rows' threads instead,
// 8 bytes a column for every warp, they alone took 1,024 cycles a tile.
//
// -lse is divided by c beforehand. This step's operands are bf16 for fp16 data too, whose
// own 16 bits end at 65504: -lse / c is as large as the largest score.
//
// 16 values of a row are two runs of 16 bytes; 8 rows' runs lie together (no swizzle). The
// scores' step and dP's share no run but one of zeros between theirs: in one run, a delta
// that is not finite would make 0 times itself a part of the scores.
constexpr int kBiasGroup = 3 * 128, kBiasForD = 128;       // bytes of 8 rows; where dP's runs begin
__device__ __forceinline__ void tc_bias_row(unsigned char *tile, int r, float a, float b, float c, float d, float e, float f) {
    uint4 *at = reinterpret_cast<uint4 *>(tile + r / 8 * kBiasGroup + r % 8 * 16);
    at[0] = make_uint4(pack2<__nv_bfloat16>(a, b), pack2<__nv_bfloat16>(c, 0.0f), 0u, 0u);
    at[8] = make_uint4(0u, 0u, 0u, 0u);
    at[16] = make_uint4(pack2<__nv_bfloat16>(d, e), pack2<__nv_bfloat16>(f, 0.0f), 0u, 0u);
}
__device__ __forceinline__ float tc_bf16(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }
// Query r's row of the operand from its pair of stat. A query without keys (or past the
// last) gets a number that leaves no weight at the smallest c, 1e-30.
__device__ __forceinline__ void tc_bias_put(unsigned char *tile, int r, const float *st, float over_c) {
    const float l = st[0] == -INFINITY ? -1e37f : st[0] * over_c, d = st[2];
    const float l1 = tc_bf16(l), l2 = tc_bf16(l - l1), d1 = tc_bf16(d), d2 = tc_bf16(d - d1);
    tc_bias_row(tile, r, l1, l2, l - l1 - l2, d1, d2, d - d1 - d2);
}

struct TcMaps {
    CUtensorMap a1, a2, x1, x2;        // rows: one or two; columns: two
};

// Block `block` of a mode.
template <typename T, int MODE, int DP, bool SHORT>
__device__ __forceinline__ void attn_tc_block(const AttnArgs &a, const TcMaps &maps, int block) {
    using K = Tc<MODE, DP, SHORT>;
    constexpr int BN = K::BN, STAGES = K::STAGES, EARLY = K::EARLY, INFO = K::INFO, HELPER = K::PARTS * 4;
    constexpr bool BF16 = TcScale<T>::forward == 0.0f, BACK = K::BACK;
    // Which operand's tile is only used for the scores, and free after them: forward's k,
    // the x1, and dq's v, the x2. The other one's stays for the second product.
    constexpr bool FIRST_EARLY = MODE == kForward;
    extern __shared__ unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *tile_a1 = base, *tile_a2 = base + K::ROW_BYTES, *tile_late = base + (BACK ? 2 : 1) * K::ROW_BYTES;
    unsigned char *tile_early = tile_late + STAGES * K::COL_BYTES;
    unsigned char *tile_stat = base + K::TILES, *tile_bias = tile_stat + STAGES * K::STAT_BYTES, *ones = tile_bias + STAGES * K::BIAS_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ones + K::ONES_BYTES);
    uint64_t *a_full = bars, *full = bars + 1, *empty = full + STAGES, *full_early = empty + STAGES, *empty_early = full_early + EARLY;
    // scores, and dP (d_); weights ready and used: P's (kGradKV: p_), and the last ones of a tile
    uint64_t *s_full = empty_early + EARLY, *s_free = s_full + 1, *d_full = s_free + 1, *d_free = d_full + 1;
    uint64_t *p_ready = d_free + 1, *p_done = p_ready + 1, *ready = p_done + 1, *done = ready + 2, *last = done + 2, *bias_full = last + 2;
    TcTile *info = reinterpret_cast<TcTile *>(bias_full + STAGES);        // [INFO]
    uint32_t *slot = reinterpret_cast<uint32_t *>(info + INFO);
    volatile uint32_t *dead = slot + 1;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    const int split = block % a.splits;
    const AttnRows w = attn_rows<MODE, kTcRows>(a, block / a.splits);
    const int64_t tiles = attn_column_tiles<MODE, BN>(a);
    const int64_t j0 = tiles * split / a.splits, j1 = tiles * (split + 1) / a.splits;

    if (warp == HELPER) {
        tmem_alloc<K::COLS>(slot);
    } else if (warp == HELPER + 1 && lane == 0) {
        bar_init(a_full, 1);
        for (int i = 0; i < STAGES; ++i) {
            bar_init(full + i, 1);
            bar_init(empty + i, 1);
        }
        for (int i = 0; i < EARLY; ++i) {
            bar_init(full_early + i, 1);
            bar_init(empty_early + i, 1);
        }
        for (int i = 0; i < STAGES; ++i) bar_init(bias_full + i, 1);
        bar_init(s_full, 1);
        bar_init(d_full, 1);
        bar_init(s_free, K::ROW_THREADS);
        bar_init(d_free, K::ROW_THREADS);
        bar_init(p_ready, K::ROW_THREADS);
        bar_init(p_done, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(ready + i, K::ROW_THREADS);
            bar_init(done + i, 1);
            bar_init(last + i, 1);
        }
        bar_init_done();
        *dead = 0u;
    }
    attn_after();
    if (MODE == kGradKV) {
        for (int i = threadIdx.x; i < kTcRows; i += K::THREADS) tc_bias_row(ones, i, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f);
        shared_to_async();
    }
    tmem_before_sync();
    __syncthreads();
    tmem_after_sync();
    const uint32_t tmem = *slot;

    if (warp >= HELPER) {
        fewer_registers<K::REGS_OTHER>();
        if (warp == HELPER + 1) {
            // -------------------------------------------- fetching
            // Each lane finds the class of one of the next 32 column tiles.
            int it = 0;
            Ring<STAGES> st;
            Ring<EARLY> se;
            bool ok = true;
            for (int64_t j = j0; j < j1 && ok; j += 32) {
                int its_pos = 0, its_head = 0, its_cls = 0;
                if (j + lane < j1) {
                    attn_columns<MODE, BN>(a, w, j + lane, &its_pos, &its_head);
                    its_cls = attn_class<MODE, BN>(a, w, its_pos, its_head);
                }
                for (uint32_t left = __ballot_sync(0xffffffffu, its_cls != 0); left && ok; left &= left - 1) {
                    const int from = __ffs(left) - 1;
                    const int pos = __shfl_sync(0xffffffffu, its_pos, from), head = __shfl_sync(0xffffffffu, its_head, from);
                    const int cls = __shfl_sync(0xffffffffu, its_cls, from);
                    if (it == 0) {
                        bar_expect(a_full, (BACK ? 2 : 1) * (K::PITCH * K::PANELS) * (kTcRows / w.pack * w.pack));
                        for (int p = 0; p < K::PANELS; ++p) {
                            tma_load(tile_a1 + p * kTcRows * K::PITCH, &maps.a1, 64 * p, w.head, w.pos, w.b, a_full);
                            if (BACK) tma_load(tile_a2 + p * kTcRows * K::PITCH, &maps.a2, 64 * p, w.head, w.pos, w.b, a_full);
                        }
                    }
                    ok = bar_wait(empty_early + se.at, se.phase ^ 1u, dead, a.err);
                    if (!ok) break;
                    if (lane == 0) info[it % INFO] = {pos, head, cls};
                    __syncwarp();
                    bar_expect(full_early + se.at, K::COL_BYTES);
                    for (int p = 0; p < K::PANELS; ++p)
                        tma_load(tile_early + se.at * K::COL_BYTES + p * BN * K::PITCH, FIRST_EARLY ? &maps.x1 : &maps.x2, 64 * p, head, pos, w.b, full_early + se.at);
                    ok = bar_wait(empty + st.at, st.phase ^ 1u, dead, a.err);
                    if (!ok) break;
                    bar_expect(full + st.at, K::COL_BYTES + K::STAT_BYTES);
                    for (int p = 0; p < K::PANELS; ++p)
                        tma_load(tile_late + st.at * K::COL_BYTES + p * BN * K::PITCH, FIRST_EARLY ? &maps.x2 : &maps.x1, 64 * p, head, pos, w.b, full + st.at);
                    if (MODE == kGradKV) bulk_load(tile_stat + st.at * K::STAT_BYTES, attn_stat(a, w.b, head, pos), K::STAT_BYTES, full + st.at);
                    ++it;
                    st.next();
                    se.next();
                }
            }
            // the end, for all
            if (ok && bar_wait_all(dead, a.err, Phase{empty_early + se.at, se.phase ^ 1u}, Phase{empty + st.at, st.phase ^ 1u})) {
                if (lane == 0) info[it % INFO].cls = 0;
                __syncwarp();
                bar_arrive_one(full_early + se.at);
                bar_arrive_one(full + st.at);
            }
            if (*dead) {               // copies under way end before the block does
                uint32_t off = 0u;
                if (it > 0) bar_wait(a_full, 0, &off, nullptr);
                for (int i = it < EARLY ? 0 : it - EARLY; i < it; ++i) bar_wait(full_early + i % EARLY, (i / EARLY) & 1, &off, nullptr);
                for (int i = it < STAGES ? 0 : it - STAGES; i < it; ++i) bar_wait(full + i % STAGES, (i / STAGES) & 1, &off, nullptr);
            }
        } else if (warp == HELPER) {
            // -------------------------------------------- scores
            const int steps = (a.D + 15) / 16;
            const uint32_t a1 = desc_low(shared_at(tile_a1), 16), a2 = desc_low(shared_at(tile_a2), 16);
            const uint32_t late = desc_low(shared_at(tile_late), 16), early = desc_low(shared_at(tile_early), 16);
            const uint32_t bias_at = desc_low(shared_at(tile_bias), 128), ones_at = desc_low(shared_at(ones), 128);
            constexpr uint32_t id = mma_desc<BF16, BN, false>(), high = desc_high<K::PITCH>();
            constexpr uint32_t bias_id = mma_desc<true, BN, false>(), plain = desc_high_plain(kBiasGroup);
            constexpr int per = K::PITCH / 32;      // steps of 16 channels in a panel
            // the products of a row tile and a column tile
            auto product = [&](uint32_t d, uint32_t rows, uint32_t columns) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    if (k >= steps) break;
                    mma_shared<id, high>(d, rows + desc_step(k / per * (kTcRows * K::PITCH) + k % per * 32),
                                         columns + desc_step(k / per * (BN * K::PITCH) + k % per * 32), k > 0);
                }
            };
            bool ok = true;
            Ring<STAGES> st;
            Ring<EARLY> se;
            for (int it = 0;; ++it) {
                // The tiles are there; and the columns are free: the last scores are read, and
                // (ALIAS: these became weights) the weights that will be written over are used.
                const uint32_t last_phase = (it & 1) ^ 1u;
                const Phase tile = {full_early + se.at, se.phase}, tile2 = {BACK ? full + st.at : full_early + se.at, BACK ? st.phase : se.phase};
                const Phase tile3 = MODE == kGradKV ? Phase{bias_full + st.at, st.phase} : tile;
                const Phase free = K::SPLIT ? Phase{p_done, last_phase} : K::ALIAS ? Phase{done, last_phase} : Phase{s_free, last_phase};
                const Phase used = K::WEIGHTS == 2 ? Phase{done + (it & 1), ((it >> 1) & 1) ^ 1u} : free;
                ok = MODE == kGradKV ? bar_wait_all(dead, a.err, tile, tile2) && (info[it % INFO].cls == 0 || bar_wait(tile3.bar, tile3.parity, dead, a.err))
                   : BACK ? bar_wait_all(dead, a.err, tile, tile2) : bar_wait(tile.bar, tile.parity, dead, a.err);
                if (!ok) break;
                const bool end = info[it % INFO].cls == 0;
                if (it == 0 && !end && !bar_wait(a_full, 0, dead, a.err)) break;
                ok = K::WEIGHTS == 2 ? bar_wait_all(dead, a.err, free, used) : bar_wait(free.bar, free.parity, dead, a.err);
                if (!ok) break;
                tmem_after_sync();
                if (end) {             // not before: it would be taken for the last scores' arrival
                    bar_arrive_one(s_full);
                    break;
                }
                const uint32_t x_late = late + st.at * desc_step(K::COL_BYTES), x_early = early + se.at * desc_step(K::COL_BYTES);
                const uint32_t columns = bias_at + st.at * desc_step(K::BIAS_BYTES);
                product(tmem, a1, FIRST_EARLY ? x_early : x_late);
                if (MODE == kGradKV) mma_shared<bias_id, plain>(tmem, ones_at, columns, true);
                if (MODE == kForward) mma_commit(empty_early + se.at);
                if (!BACK || K::SPLIT) mma_commit(s_full);
                if (BACK) {
                    if (K::SPLIT) {
                        ok = bar_wait(done, last_phase, dead, a.err);
                        if (!ok) break;
                        tmem_after_sync();
                    }
                    product(tmem + BN, a2, x_early);
                    if (MODE == kGradKV) mma_shared<bias_id, plain>(tmem + BN, ones_at + desc_step(kBiasForD), columns + desc_step(kBiasForD), true);
                    if (MODE == kGradQ) mma_commit(empty_early + se.at);
                    mma_commit(K::SPLIT ? d_full : s_full);
                }
                st.next();
                se.next();
            }
            if (!ok) {                 // MMAs under way end before the block does
                uint32_t off = 0u;
                mma_commit(last);
                bar_wait(last, 0, &off, nullptr);
            }
        } else if (warp == HELPER + 2) {
            // -------------------------------------------- second products
            const uint32_t late = desc_low(shared_at(tile_late), BN * K::PITCH), early = desc_low(shared_at(tile_early), BN * K::PITCH);
            constexpr uint32_t id = mma_desc<BF16, DP, true>(), high = desc_high<K::PITCH>();
            constexpr int PART_STEPS = K::PART / 16;
            auto product = [&](uint32_t d, uint32_t weights, uint32_t columns, bool add) {
#pragma unroll
                for (int k = 0; k < BN / 16; ++k)      // over the scores each part's weights are in its own columns
                    mma_tmem<id, high>(d, weights + (K::ALIAS ? k / PART_STEPS * K::PART + k % PART_STEPS * 8 : 8 * k), columns + desc_step(k * 16 * K::PITCH), add || k > 0);
            };
            bool ok = true;
            Ring<STAGES> st;
            Ring<EARLY> se;
            for (int it = 0;; ++it) {
                ok = MODE == kGradKV ? bar_wait_all(dead, a.err, Phase{full + st.at, st.phase}, Phase{full_early + se.at, se.phase})
                                     : bar_wait(full + st.at, st.phase, dead, a.err);
                if (!ok || !info[it % INFO].cls) break;
                const uint32_t x_late = late + st.at * desc_step(K::COL_BYTES), x_early = early + se.at * desc_step(K::COL_BYTES), acc = tmem + K::ACC;
                // weights: P, then dS
                const uint32_t p = tmem + (K::ALIAS ? 0 : K::SCORES + (K::WEIGHTS == 2 ? (it & 1) * K::WIDE : 0));
                const uint32_t ds = MODE != kGradKV ? p : K::ALIAS ? p + BN : p + BN / 2;
                if (K::SPLIT) {
                    ok = bar_wait(p_ready, it & 1, dead, a.err);
                    if (!ok) break;
                    tmem_after_sync();
                    product(acc, p, x_early, it > 0);
                    mma_commit(p_done);
                }
                ok = bar_wait(tc_bar<K::WEIGHTS>(ready, it), tc_phase<K::WEIGHTS>(it), dead, a.err);
                if (!ok) break;
                tmem_after_sync();
                if (MODE == kGradKV && !K::SPLIT) product(acc, p, x_early, it > 0);
                product(acc + (MODE == kGradKV ? DP : 0), ds, x_late, it > 0);
                if (MODE == kGradKV) mma_commit(empty_early + se.at);    // dP, which reads it too, is there
                mma_commit(empty + st.at);
                mma_commit(tc_bar<K::WEIGHTS>(done, it));  // last: the block ends after it has arrived
                st.next();
                se.next();
            }
            if (!ok) {
                uint32_t off = 0u;
                mma_commit(last + 1);
                bar_wait(last + 1, 0, &off, nullptr);
            }
        } else if (MODE == kGradKV) {
            // -------------------------------------------- the queries' statistics as an operand
            const float over_c = 1.0f / a.c;
            Ring<STAGES> st;
            for (int it = 0;; ++it, st.next()) {
                if (!bar_wait(full + st.at, st.phase, dead, a.err) || !info[it % INFO].cls) break;
                for (int i = lane; i < BN; i += 32)
                    tc_bias_put(tile_bias + st.at * K::BIAS_BYTES, i, reinterpret_cast<const float *>(tile_stat + st.at * K::STAT_BYTES) + i / 2 * 4 + i % 2, over_c);
                shared_to_async();
                __syncwarp();
                bar_arrive_one(bias_full + st.at);
            }
        }
        __syncwarp();
    } else {
        more_registers<K::REGS_ROW>();
        // ------------------------------------------------ one row a thread
        const int part = warp / 4, r = threadIdx.x % 128;  // columns PART part on of each tile
        const bool valid = w.valid(r);
        const bool any_valid = w.valid(r & ~31);           // of this warp's rows
        const uint32_t mine = tmem + ((uint32_t)(r & ~31) << 16), at_acc = mine + K::ACC;
        constexpr int PART = K::PART;
        const int rpos = w.row_pos(valid ? r : 0), rhead = w.row_head(valid ? r : 0);
        const float c = a.c;
        float ds_scale = 1.0f;
        if (BACK && !BF16) ds_scale = tc_ds_scale<MODE>(a, w, MODE == kGradQ && valid ? tc_square(attn_at<T>(a, a.go, w.b, rpos, rhead), a.D) : 0.0f);
        constexpr float up = TcScale<T>::forward;
        float top = -INFINITY, sum = 0.0f, lse2 = 0.0f, delta = 0.0f;    // backward: negative, as in stat
        if (MODE == kGradQ && valid) {
            const float *st = attn_stat(a, w.b, rhead, rpos);
            lse2 = st[0];
            delta = st[2];
        }
        const uint32_t *words = MODE == kGradKV ? nullptr : attn_word_row<MODE>(a, w.b, rhead, rpos);

        // after a wait that ran out (ok false) the group's threads go on to their results'
        // barriers
        bool ok = true;
        int it = 0;
        Ring<STAGES> st;
        for (;; ++it, st.next()) {
            const uint32_t at_p = mine + (K::ALIAS ? PART * part : K::SCORES + (K::WEIGHTS == 2 ? it % 2 * K::WIDE : 0) + PART / 2 * part);
            const uint32_t at_ds = MODE != kGradKV ? at_p : K::ALIAS ? at_p + BN : at_p + BN / 2;
            // a mask's words are asked for before the scores are there (their tile's barrier moves
            // on only after this tile's second product)
            ok = a.classes ? bar_wait(full + st.at, st.phase, dead, a.err) : bar_wait(s_full, it & 1, dead, a.err);
            if (!ok) break;
            const TcTile tile = info[it % INFO];
            const int cls = tile.cls;
            if (!cls) break;
            uint32_t bits[PART / 32];
            if (cls != 2) {
                if (MODE == kGradKV) words = attn_word_row<MODE>(a, w.b, tile.head, rpos);
#pragma unroll
                for (int i = 0; i < PART / 32; ++i) bits[i] = attn_word<MODE>(a, words, tile.pos + PART * part + 32 * i);
            }
            if (a.classes) ok = bar_wait(s_full, it & 1, dead, a.err);
            if (!ok) break;
            tmem_after_sync();
            // the row's scores, and dP beside them unless it comes later
            uint32_t v[PART], dp[BACK ? PART : 1];
            if (any_valid) {
                if constexpr (BACK && !K::SPLIT) tmem_read_two<PART>(v, dp, mine + PART * part, mine + BN + PART * part);
                else tmem_read<PART>(v, mine + PART * part);
            }
            if (!K::ALIAS) {
                tmem_before_sync();
                bar_arrive(s_free);
            }
            if (cls != 2) {            // p, and with it ds unless dP is not finite, will be 0
#pragma unroll
                for (int k = 0; k < PART; ++k)
                    if (!((bits[k / 32] >> (k % 32)) & 1u)) v[k] = 0xff800000u;
            }
            // The weights' columns are free. Forward waits here, backward after its arithmetic; waited
            // for after the maximum, 4096 x 4096 of 64 channels take 195 us, not 174.
            if (MODE == kForward && K::WEIGHTS == 1 && it > 0) {
                ok = bar_wait(tc_bar<K::WEIGHTS>(done, it - 1), tc_phase<K::WEIGHTS>(it - 1), dead, a.err);
                if (!ok) break;
                tmem_after_sync();
            }
            const float2 c2 = make_float2(c, c);
            auto pair = [](const uint32_t *x) { return make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])); };
            uint32_t out[MODE == kGradKV ? PART / 2 : 1], out2[BACK ? PART / 2 : 1];     // weights: P, dS
            if (any_valid && MODE == kForward) {
                float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < PART; k += 2) most[k / 2 % 4] = max3(most[k / 2 % 4], pair(v + k).x, pair(v + k).y);
                const float high = max3(fmaxf(most[0], most[1]), most[2], most[3]);
                // The weights are relative to `top`, which follows the maximum only when that has
                // grown by more than 2^8: then what was summed is scaled down.
                const bool grow = top == -INFINITY ? high > -INFINITY : (high - top) * c > 8.0f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = !grow ? 1.0f : top == -INFINITY ? 0.0f : ex2((top - high) * c);
                    if (grow) top = high;
                    sum *= f;
                    if (it > 0) {
                        if (K::WEIGHTS != 1) ok = bar_wait(tc_bar<K::WEIGHTS>(done, it - 1), tc_phase<K::WEIGHTS>(it - 1), dead, a.err);
                        tmem_after_sync();
#pragma unroll 1
                        for (int i = 0; ok && i < DP; i += 16) {
                            uint32_t o[16];
                            tmem_read<16>(o, at_acc + i);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_store16(at_acc + i, o);
                        }
                    }
                }
                const float ref = tc_reference(top, c, up);
                const float2 ref2 = make_float2(-ref, -ref);
                float2 sums[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int i = 0; i < PART; i += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 x = __ffma2_rn(pair(v + i + k), c2, ref2);
                        const float2 p = make_float2(ex2(x.x), ex2(x.y));
                        sums[k / 2 % 2] = __fadd2_rn(sums[k / 2 % 2], p);
                        w[k / 2] = pack2<T>(p.x, p.y);
                    }
                    tmem_store16(at_p + i / 2, w);
                }
                sum += (sums[0].x + sums[1].x) + (sums[0].y + sums[1].y);
            }
            if constexpr (BACK) {
                const float2 l2 = make_float2(lse2, lse2), e2 = make_float2(delta, delta), one = make_float2(ds_scale, ds_scale);
                auto probability = [&](int k) {
                    const float2 x = MODE == kGradKV ? __fmul2_rn(pair(v + k), c2) : __ffma2_rn(pair(v + k), c2, l2);
                    return make_float2(ex2(x.x), ex2(x.y));
                };
                auto slope = [&](float2 p, int k) {
                    const float2 d = __fmul2_rn(p, MODE == kGradKV ? pair(dp + k) : __fadd2_rn(pair(dp + k), e2));
                    return BF16 ? d : __fmul2_rn(d, one);
                };
                if constexpr (K::SPLIT) {
                    if (any_valid) {   // p in place of the scores
#pragma unroll
                        for (int k = 0; k < PART; k += 2) {
                            const float2 p = probability(k);
                            out[k / 2] = pack2<T>(p.x, p.y);
                            v[k] = __float_as_uint(p.x);
                            v[k + 1] = __float_as_uint(p.y);
                        }
                        tmem_store<PART / 2>(at_p, out);
                        tmem_wait_store();
                    }
                    tmem_before_sync();
                    bar_arrive(p_ready);
                    ok = bar_wait(d_full, it & 1, dead, a.err);
                    if (!ok) break;
                    tmem_after_sync();
                    if (any_valid) {
                        tmem_read<PART>(dp, mine + BN + PART * part);
#pragma unroll
                        for (int k = 0; k < PART; k += 2) {
                            const float2 d = slope(pair(v + k), k);
                            out2[k / 2] = pack2<T>(d.x, d.y);
                        }
                    }
                } else if (any_valid) {
#pragma unroll
                    for (int k = 0; k < PART; k += 2) {
                        const float2 p = probability(k), d = slope(p, k);
                        if (MODE == kGradKV) out[k / 2] = pack2<T>(p.x, p.y);
                        out2[k / 2] = pack2<T>(d.x, d.y);
                    }
                }
            }
            if (BACK && K::WEIGHTS == 1 && it > 0) {
                ok = bar_wait(tc_bar<K::WEIGHTS>(done, it - 1), tc_phase<K::WEIGHTS>(it - 1), dead, a.err);
                tmem_after_sync();
            }
            if (!ok) break;
            if (any_valid) {
                if constexpr (MODE == kGradKV && !K::SPLIT) tmem_store<PART / 2>(at_p, out);
                if constexpr (BACK) tmem_store<PART / 2>(at_ds, out2);
                tmem_wait_store();
            }
            tmem_before_sync();
            bar_arrive(tc_bar<K::WEIGHTS>(ready, it));
        }

        // ------------------------------------------------ results
        if (ok && it > 0) ok = bar_wait(tc_bar<K::WEIGHTS>(done, it - 1), tc_phase<K::WEIGHTS>(it - 1), dead, a.err);
        tmem_after_sync();
        // column tiles of the block; a wait that ran out leaves NaN, not what was in the output
        const bool lost = !__all_sync(0xffffffffu, ok && !*dead);
        const int count = lost ? 0 : it;
        const float none = lost ? __int_as_float(0x7fffffff) : 0.0f;
        if (lost) sum = none;
        if (any_valid) {
            const int64_t row = MODE == kGradKV ? ((int64_t)w.b * a.S + rpos) * a.N + rhead : ((int64_t)w.b * a.Q + rpos) * a.M + rhead;
            const float ref = tc_reference(top, c, up);
            const float down = BACK ? ex2(-TcScale<T>::backward) : 1.0f;   // of P; of dS also 1 / ds_scale
            const float down_ds = down / ds_scale;
            if (MODE == kForward && valid) {
                if (a.splits > 1) {
                    float *ml = a.part + (int64_t)a.splits * a.part_rows * a.D + 2 * ((int64_t)split * a.part_rows + row);
                    ml[0] = sum == 0.0f ? -INFINITY : ref;
                    ml[1] = sum;
                } else if (a.lse) {
                    attn_put_lse(a, w.b, rhead, rpos, sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * kLn2);
                }
            }
            const float over = sum == 0.0f ? 0.0f : 1.0f / sum;
            uint32_t open = 0u;        // of this group's chunks, those that are not finite
            // 32 channels of a result at a time, shared among the groups
#pragma unroll 1
            for (int q = part; q < K::RESULTS * (DP / 32); q += K::PARTS) {
                const int which = q / (DP / 32), d0 = q % (DP / 32) * 32;
                const float g = MODE == kForward ? 1.0f : MODE == kGradQ || which ? down_ds : down;
                const float f = MODE == kForward ? over : g * (MODE == kGradQ || which ? a.scale : 1.0f);
                uint32_t o[32];
                float v[32];
                if (count > 0) tmem_read<32>(o, at_acc + 32 * q);
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = count > 0 ? __uint_as_float(o[k]) : none;
                if (a.classes && !lost) {
                    bool finite = true;
#pragma unroll
                    for (int k = 0; k < 32; ++k) finite = finite && isfinite(v[k]);
                    if (valid && !finite) open |= 1u << q;
                }
                if (valid) tc_store<T, MODE>(a, row, split, which, d0, v, f, g);
            }
            if (__any_sync(0xffffffffu, open)) {
                const bool again = attn_spoiled<T, MODE, BN>(a, w, open ? r : -1, j0, j1, MODE == kForward && !isfinite(sum));
                for (uint32_t bad = __ballot_sync(0xffffffffu, again); bad; bad &= bad - 1) {
                    const int from = __ffs(bad) - 1;
                    float e1[4], e2[4];
                    const float m2 = __shfl_sync(0xffffffffu, ref, from), over_from = __shfl_sync(0xffffffffu, over, from);
                    const uint32_t chunks = __shfl_sync(0xffffffffu, open, from);
                    attn_exact_row<T, MODE, BN>(a, w, (r & ~31) + from, j0, j1, m2, e1, e2);
                    __syncwarp();      // in place of what its lane has stored
#pragma unroll
                    for (int i = 0; i < K::RESULTS * (DP / 32); ++i) {
                        const int which = i / (DP / 32), c = i % (DP / 32), at = 32 * c + lane;
                        if (!((chunks >> i) & 1u) || at >= a.D) continue;
                        const bool of_ds = MODE == kGradQ || which;
                        attn_store<T, MODE>(a, w, (r & ~31) + from, split, which, at, of_ds ? e2[c] : e1[c],
                                            MODE == kForward ? over_from : of_ds ? a.scale : 1.0f);
                    }
                }
            }
        }
        tmem_before_sync();
    }
    __syncthreads();
    if (warp == HELPER) {
        tmem_after_sync();
        tmem_free<K::COLS>(tmem);
    }
}

template <typename T, int MODE, int DP, bool SHORT>
__global__ void __launch_bounds__(Tc<MODE, DP, SHORT>::THREADS, Tc<MODE, DP, SHORT>::BLOCKS)
attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ TcMaps maps) {
    attn_tc_block<T, MODE, DP, SHORT>(a, maps, blockIdx.x);
}

// Both gradients' blocks in one launch: neither needs the other's results, and the last ones
// of one kind leave no SM idle. The kind whose blocks take longer is first (`first` blocks of
// it). One launch after the other: 17.3 us instead of 11.1 for 300 queries and keys of 2 x 8
// heads of 32, 511 instead of 502 for 4,096 of 32 heads of 64; the queries' first there: 510;
// the keys' first for 60 queries of 4 x 8 heads of 32 over 600 keys: 17.5 instead of 14.4.
template <typename T, int DP>
__global__ void __launch_bounds__(Tc<kGradQ, DP, false>::THREADS, 1)
attn_tc_back_kernel(const __grid_constant__ AttnArgs q, const __grid_constant__ TcMaps q_maps, int first, bool keys_first,
                    const __grid_constant__ AttnArgs kv, const __grid_constant__ TcMaps kv_maps) {
    static_assert((int)Tc<kGradQ, DP, false>::THREADS == (int)Tc<kGradKV, DP, false>::THREADS, "one launch");
    const bool early = (int)blockIdx.x < first;
    const int block = early ? blockIdx.x : blockIdx.x - first;
    if (early == keys_first) attn_tc_block<T, kGradKV, DP, false>(kv, kv_maps, block);
    else attn_tc_block<T, kGradQ, DP, false>(q, q_maps, block);
}

// ------------------------------------------------------------------ launch

// A map of boxes of `heads` heads and `positions` positions.
template <int MODE, int DP, bool SHORT>
cudaError_t tc_map(CUtensorMap *map, const AttnTensor &t, const AttnArgs &a, int len, int heads, int box_heads, int box_positions,
                   bool bf16) {
    using K = Tc<MODE, DP, SHORT>;
    const cuuint64_t dense = (cuuint64_t)a.D * 2;
    const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)heads, (cuuint64_t)len, (cuuint64_t)a.B};
    const cuuint64_t strides[3] = {heads > 1 ? (cuuint64_t)t.head * 2 : dense, len > 1 ? (cuuint64_t)t.pos * 2 : dense,
                                   a.B > 1 ? (cuuint64_t)t.batch * 2 : dense};
    const cuuint32_t box[4] = {(cuuint32_t)K::PANEL, (cuuint32_t)box_heads, (cuuint32_t)box_positions, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const CUresult r = encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                              const_cast<void *>(t.p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              K::PITCH == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The maps of a mode's tensors. No columns: the maps are of what is there, and nothing is
// fetched.
template <typename T, int MODE, int DP, bool SHORT> cudaError_t tc_maps(TcMaps *maps, const AttnArgs &a) {
    using K = Tc<MODE, DP, SHORT>;
    constexpr bool bf16 = TcScale<T>::forward == 0.0f;
    cudaError_t e;
    const bool none = MODE == kGradKV ? a.Q == 0 : a.S == 0;
    if (MODE == kGradKV) {
        const AttnTensor &x1 = none ? a.k : a.q, &x2 = none ? a.v : a.go;
        const int len = none ? a.S : a.Q, heads = none ? a.N : a.M;
        if ((e = tc_map<MODE, DP, SHORT>(&maps->a1, a.k, a, a.S, a.N, 1, kTcRows, bf16)) != cudaSuccess ||
            (e = tc_map<MODE, DP, SHORT>(&maps->a2, a.v, a, a.S, a.N, 1, kTcRows, bf16)) != cudaSuccess ||
            (e = tc_map<MODE, DP, SHORT>(&maps->x1, x1, a, len, heads, 1, K::BN, bf16)) != cudaSuccess)
            return e;
        return tc_map<MODE, DP, SHORT>(&maps->x2, x2, a, len, heads, 1, K::BN, bf16);
    }
    const AttnTensor &x1 = none ? a.q : a.k, &x2 = none ? a.q : a.v;
    const int len = none ? a.Q : a.S, heads = none ? a.M : a.N;
    if ((e = tc_map<MODE, DP, SHORT>(&maps->a1, a.q, a, a.Q, a.M, a.pack, kTcRows / a.pack, bf16)) != cudaSuccess ||
        (e = tc_map<MODE, DP, SHORT>(&maps->x1, x1, a, len, heads, 1, K::BN, bf16)) != cudaSuccess ||
        (e = tc_map<MODE, DP, SHORT>(&maps->x2, x2, a, len, heads, 1, K::BN, bf16)) != cudaSuccess)
        return e;
    maps->a2 = maps->a1;
    if (MODE != kGradQ) return cudaSuccess;
    return tc_map<MODE, DP, SHORT>(&maps->a2, a.go, a, a.Q, a.M, a.pack, kTcRows / a.pack, bf16);
}

template <typename T, int MODE, int DP, bool SHORT>
cudaError_t launch_tc_d(const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    using K = Tc<MODE, DP, SHORT>;
    TcMaps maps;
    cudaError_t e = tc_maps<T, MODE, DP, SHORT>(&maps, a);
    if (e != cudaSuccess) return e;
    auto *kernel = attn_tc_kernel<T, MODE, DP, SHORT>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SHARED);
    if (e != cudaSuccess) return e;
    return launch_after(a.chained, kernel, blocks, K::THREADS, K::SHARED, stream, a, maps);
}
template <typename T>
cudaError_t launch_tc(const AttnArgs &a, int64_t blocks, cudaStream_t stream) {
    return a.D <= 32 ? launch_tc_d<T, kForward, 32, false>(a, blocks, stream)
         : a.D <= 64 ? launch_tc_d<T, kForward, 64, false>(a, blocks, stream)
                     : launch_tc_d<T, kForward, 128, false>(a, blocks, stream);
}

template <typename T, int DP>
cudaError_t launch_tc_back_d(const AttnArgs &q, int64_t q_blocks, const AttnArgs &kv, int64_t kv_blocks, cudaStream_t stream) {
    using Q = Tc<kGradQ, DP, false>;
    using KV = Tc<kGradKV, DP, false>;
    constexpr int bytes = Q::SHARED > KV::SHARED ? Q::SHARED : KV::SHARED;
    TcMaps q_maps = {}, kv_maps = {};
    cudaError_t e = q_blocks > 0 ? tc_maps<T, kGradQ, DP, false>(&q_maps, q) : cudaSuccess;
    if (e == cudaSuccess && kv_blocks > 0) e = tc_maps<T, kGradKV, DP, false>(&kv_maps, kv);
    if (e != cudaSuccess) return e;
    auto *kernel = attn_tc_back_kernel<T, DP>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    // by column tiles a block; the keys' take a third longer
    const int64_t q_walk = attn_column_tiles<kGradQ, Q::BN>(q) / q.splits, kv_walk = attn_column_tiles<kGradKV, KV::BN>(kv) / kv.splits;
    const bool keys_first = 4 * kv_walk >= 3 * q_walk;
    return launch_after(true, kernel, q_blocks + kv_blocks, Q::THREADS, bytes, stream, q, q_maps, (int)(keys_first ? kv_blocks : q_blocks), keys_first, kv, kv_maps);
}
// The gradients; no blocks of a kind that is not wanted. The small blocks of few queries
// (tc_short) have a launch of their own.
template <typename T>
cudaError_t launch_tc_back(const AttnArgs &q, int64_t q_blocks, const AttnArgs &kv, int64_t kv_blocks, cudaStream_t stream) {
    if (q_blocks == 0 && tc_short(kv))
        return kv.D <= 32 ? launch_tc_d<T, kGradKV, 32, true>(kv, kv_blocks, stream) : launch_tc_d<T, kGradKV, 64, true>(kv, kv_blocks, stream);
    return q.D <= 32 ? launch_tc_back_d<T, 32>(q, q_blocks, kv, kv_blocks, stream)
         : q.D <= 64 ? launch_tc_back_d<T, 64>(q, q_blocks, kv, kv_blocks, stream)
                     : launch_tc_back_d<T, 128>(q, q_blocks, kv, kv_blocks, stream);
}

}  // namespace msda
