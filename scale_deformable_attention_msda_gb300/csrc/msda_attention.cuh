// Dense attention's shared pieces: arguments, the packed mask, and rows in
// which something is not finite.
//
// Forward and backward are one scheme in three modes. A block holds a tile of
// rows and walks tiles of columns; every score is computed where it is used and
// none is stored:
//
// kForward   rows are queries, columns keys:   out  = sum_j p_ij v_j
// kGradQ     rows are queries, columns keys:   dq   = scale sum_j ds_ij k_j
// kGradKV    rows are keys, columns queries:   dv   = sum_i p_ij dO_i
//                                              dk   = scale sum_i ds_ij q_i
// with s_ij = q_i k_j (raw), p_ij = exp2(c s_ij - log2 of the row's sum), c =
// scale log2(e), and ds_ij = p_ij (dO_i v_j - delta_i), delta_i = dO_i out_i.
// The backward computes the scores twice, once for dq and once for dk and dv: 7
// products in place of 5, and in return no sum is added up in memory by atomics
// in an order that changes.
//
// Few queries leave a tile of rows empty, so query heads that share a key head
// lie in it together (pack heads a position); and when the row tiles do not fill
// the SMs, each tile's columns are split over several blocks whose results a
// second kernel joins.
#pragma once

#include "msda_common.cuh"

namespace msda {

enum AttnMode { kForward = 0, kGradQ = 1, kGradKV = 2 };

constexpr int kAttnMaxD = 128;
constexpr int kAttnGranule = 64;       // queries and keys of one class of the mask
constexpr float kLog2e = 1.4426950408889634f;
// fp16 holds what lies between 2^-24 and 65504: the backward's probabilities are scaled
// by 2^14, the forward's weights, at most 2^8, by 2^7.
constexpr float kHalfUp = 14.0f, kHalfWeightUp = 7.0f;
constexpr float kLn2 = 0.6931471805599453f;

// A tensor of positions and heads: strides in elements, and its extents.
struct AttnTensor {
    const void *p;
    int64_t batch, pos, head;
    int len, heads;
};

// The mask as bits, one word for 32 columns; strides in words, 0 repeats.
struct AttnBits {
    const uint32_t *p;                 // NULL: every pair is allowed
    int64_t batch, head, row;
    int word;
};

struct AttnArgs {
    AttnTensor q, k, v, o, go;         // o, go: out and its gradient (backward)
    void *out, *gq, *gk, *gv;
    void *rest;                        // what out's rounding left, of out's type and shape; NULL: none
    float *lse;                        // (B, M, Q); forward: may be NULL
    // backward: (B, M, stat_row / 2, 4), for two queries each -lse in the exponent's
    // units, plus `up`, and -delta; past the last query -infinity and 0
    float *stat;
    int stat_row;                      // queries in a row of stat: Q up to a multiple of 128, the
                                       // longest tile's
    float up;                          // fp16 backward: its probabilities are scaled by 2^up
    // fp16 backward: of each batch entry and key head, partial maxima of |dO_i|^2 and
    // |v_j|^2 (norms each, see attn_delta_kernel); NULL for other types
    float *norm_do, *norm_v;
    int norms;
    AttnBits by_query, by_key;         // rows are queries (columns keys), and the other way
    const uint8_t *classes;            // of granules: 0 empty, 1 mixed, 2 all allowed
    int64_t class_batch, class_head;
    int class_row;                     // granules of keys in a row of classes; 0: one row for all
    int B, Q, S, M, N, D, G;           // G = M / N
    int pack;                          // query heads that lie in a row tile together: 1 or G
    float scale, c;
    int splits;                        // blocks that share a row tile's columns (this mode)
    float *part;                       // splits > 1: (splits, rows, D) sums, then (splits, rows, 2)
                                       // maximum and sum (forward); gradients of keys twice
    int64_t part_rows;                 // rows of this mode's results
    unsigned *err;                     // device word of range faults and of waits that ran out
    // The kernels of one call follow each other in one stream, each started while the one
    // before it ends (see attn_after). chained: there is one before.
    bool chained;
};

// Between kernels of one call: what follows sees all that the kernel before has written,
// and the next kernel may be started (it waits here itself). Saves its start behind the
// end of the one before: 1 to 3 us a kernel.
__device__ __forceinline__ void attn_after() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Checked build: whether i is one of n; a fault otherwise. Always true in the normal build.
__device__ __forceinline__ bool attn_ok(const AttnArgs &a, int64_t i, int64_t n) {
#ifdef MSDA_CHECKED
    if (i >= 0 && i < n) return true;
    if (a.err) atomicOr(a.err, 1u);
    return false;
#else
    return true;
#endif
}

// A row of a tensor (checked build: its first in place of one that it does not have).
template <typename T>
__device__ __forceinline__ const T *attn_at(const AttnArgs &a, const AttnTensor &t, int b, int pos, int head) {
    const T *first = static_cast<const T *>(t.p);
    return attn_ok(a, b, a.B) && attn_ok(a, pos, t.len) && attn_ok(a, head, t.heads) ? first + b * t.batch + pos * t.pos + head * t.head : first;
}
__device__ __forceinline__ void attn_put_lse(const AttnArgs &a, int b, int head, int pos, float lse) {
    const int64_t at = ((int64_t)b * a.M + head) * a.Q + pos;
    if (attn_ok(a, at, (int64_t)a.B * a.M * a.Q)) a.lse[at] = lse;
}

// Where a row tile's rows are. FWD and DQ: `pack` heads a position.
struct AttnRows {
    int b, head, pos, count;           // first head (of queries, or of keys) and position; positions
    int pack;
    __device__ __forceinline__ bool valid(int r) const { return r < count * pack; }
    // (a division takes 20 instructions)
    __device__ __forceinline__ int row_pos(int r) const { return pos + (pack == 1 ? r : r / pack); }
    __device__ __forceinline__ int row_head(int r) const { return head + (pack == 1 ? 0 : r % pack); }
};

// Row tile number `t` of tiles of R rows.
template <int MODE, int R>
__device__ __forceinline__ AttnRows attn_rows(const AttnArgs &a, int t) {
    AttnRows w;
    w.pack = MODE == kGradKV ? 1 : a.pack;
    const int per = R / w.pack, len = MODE == kGradKV ? a.S : a.Q;
    const int heads = MODE == kGradKV ? a.N : a.M / w.pack, tiles = (len + per - 1) / per;
    w.pos = t % tiles * per;
    w.count = min(per, len - w.pos);
    t /= tiles;
    w.head = t % heads * w.pack;
    w.b = t / heads;
    return w;
}

// Column tiles of C columns that a row tile walks.
template <int MODE, int C> __host__ __device__ __forceinline__ int64_t attn_column_tiles(const AttnArgs &a) {
    return MODE == kGradKV ? (int64_t)a.G * ((a.Q + C - 1) / C) : (a.S + C - 1) / C;
}
// The first position of column tile j and its head (of keys, or of queries).
template <int MODE, int C>
__device__ __forceinline__ void attn_columns(const AttnArgs &a, const AttnRows &w, int64_t j, int *pos, int *head) {
    if (MODE == kGradKV) {
        const int tiles = (a.Q + C - 1) / C;
        *pos = (int)(j % tiles) * C;
        *head = w.head * a.G + (int)(j / tiles);
    } else {
        *pos = (int)j * C;
        *head = w.head / a.G;
    }
}

// What the mask leaves of a row tile and a column tile: 0 nothing, 2 all pairs,
// 1 some, or columns past the end. R: positions that the row tile holds.
template <int MODE, int C>
__device__ __forceinline__ int attn_class(const AttnArgs &a, const AttnRows &w, int pos, int head) {
    const int len = MODE == kGradKV ? a.Q : a.S;
    const int whole = pos + C <= len ? 2 : 1;
    // keys past the end are masked by bits; queries past it have no weight
    if (!a.classes) return MODE == kGradKV ? 2 : whole;
    const int q0 = MODE == kGradKV ? pos : w.pos, qn = MODE == kGradKV ? min(C, a.Q - pos) : w.count;
    const int k0 = MODE == kGradKV ? w.pos : pos, kn = MODE == kGradKV ? w.count : min(C, a.S - pos);
    const int h0 = MODE == kGradKV ? head : w.head, hn = MODE == kGradKV ? 1 : w.pack;
    bool any = false, all = true;
    for (int h = h0; h < h0 + (a.class_head ? hn : 1); ++h) {
        const uint8_t *c = a.classes + w.b * a.class_batch + h * a.class_head;
        const int last = a.class_row ? (q0 + qn - 1) / kAttnGranule : 0;
        for (int i = a.class_row ? q0 / kAttnGranule : 0; i <= last; ++i)
            for (int j = k0 / kAttnGranule; j <= (k0 + kn - 1) / kAttnGranule; ++j) {
                const int v = c[(int64_t)i * a.class_row + j];
                any |= v != 0;
                all &= v == 2;
            }
    }
    return !any ? 0 : all && (MODE == kGradKV || whole == 2) ? 2 : 1;
}

// Bits of columns pos + 32 i to pos + 32 i + 31 of one row (pos a multiple of 32).
template <int MODE>
__device__ __forceinline__ uint32_t attn_word(const AttnArgs &a, const uint32_t *row, int at) {
    if (MODE == kGradKV) return !row ? 0xffffffffu : at < a.Q ? row[(int64_t)(at >> 5) * a.by_key.word] : 0u;
    if (row) return at < a.S ? row[at >> 5] : 0u;
    const int left = a.S - at;
    return left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
}
// The words of a row (rows are queries, or keys), NULL without a mask. head: of queries.
template <int MODE>
__device__ __forceinline__ const uint32_t *attn_word_row(const AttnArgs &a, int b, int head, int pos) {
    const AttnBits &m = MODE == kGradKV ? a.by_key : a.by_query;
    return m.p ? m.p + b * m.batch + head * m.head + pos * m.row : nullptr;
}

// log2 of a query's sum, as the scores' exponent needs it: a query without keys
// (or past the end) gets infinity, and with it p = 0; one with an infinite score NaN.
__device__ __forceinline__ float attn_lse2(float lse) {
    return lse == -INFINITY ? INFINITY : lse == INFINITY ? __int_as_float(0x7fffffff) : lse * kLog2e;
}

// A query's pair of stat.
__device__ __forceinline__ float *attn_stat(const AttnArgs &a, int b, int head, int pos) {
    return a.stat + ((int64_t)b * a.M + head) * a.stat_row * 2 + (pos >> 1) * 4 + (pos & 1);
}

// What lies in a masked place may be anything. Its score and its weight are replaced, but
// a product of the weight 0 with NaN or infinity is NaN. So a row whose sums are not finite
// is computed again from its allowed pairs alone (attn_exact_row), if a masked pair may be
// the cause and the allowed ones would not make all of it NaN anyway (attn_spoiled). Where
// only allowed places hold what is not finite, as in a step whose gradients overflowed, that
// search is all that such a row costs.

// A number that is finite and whose products with another such, summed over the channels, are.
constexpr float kAttnTame = 0x1p60f;
template <typename T> __device__ __forceinline__ void attn_survey(const T *row, int D, bool &tame, bool &finite) {
    constexpr int V = 16 / sizeof(T);
    float most = 0.0f;
    bool number = true;
    for (int d = 0; d < D; d += V) {
        float x[V];
        unpack16<T>(x, ldg16(row + d));
#pragma unroll
        for (int k = 0; k < V; ++k) {
            most = fmaxf(most, fabsf(x[k]));
            number = number && x[k] == x[k];
        }
    }
    tame = number && most < kAttnTame;
    finite = number && most < INFINITY;
}

// For a whole warp, each lane a row r of its own (below zero: none): whether it has to be
// computed again. The lanes look at 32 columns at a time, one each, and tell one another.
// lost: the allowed pairs make all of the row NaN.
template <typename T, int MODE, int C>
__device__ __noinline__ bool attn_spoiled(const AttnArgs &a, const AttnRows &w, int r, int64_t j0, int64_t j1, bool lost) {
    const int lane = threadIdx.x & 31;
    const int pos = w.row_pos(r < 0 ? 0 : r), head = w.row_head(r < 0 ? 0 : r);
    bool tame = true, finite = true;   // what of the row goes into its pairs' dP
    if (MODE != kForward && r >= 0) {
        attn_survey<T>(MODE == kGradQ ? attn_at<T>(a, a.go, w.b, pos, head) : attn_at<T>(a, a.v, w.b, pos, head), a.D, tame, finite);
        if (MODE == kGradQ) {
            const float *st = attn_stat(a, w.b, head, pos);
            finite = finite && st[0] < INFINITY && isfinite(st[2]);            // st[0] is -infinity without keys
            tame = tame && finite;
        }
    }
    bool allowed = false, masked = false, cause = false;
    lost = lost || r < 0;
    for (int64_t j = j0; j < j1; ++j) {
        int cpos, chead;
        attn_columns<MODE, C>(a, w, j, &cpos, &chead);
        if (!attn_class<MODE, C>(a, w, cpos, chead)) continue;
        const uint32_t *words = attn_word_row<MODE>(a, w.b, MODE == kGradKV ? chead : head, pos);
        for (int c0 = 0; c0 < C; c0 += 32) {
            const int at = cpos + c0 + lane, len = MODE == kGradKV ? a.Q : a.S;
            if (cpos + c0 >= len) break;
            bool mild = true, number = true, unused;
            if (at < len) {
                attn_survey<T>(MODE == kGradKV ? attn_at<T>(a, a.go, w.b, at, chead) : attn_at<T>(a, a.v, w.b, at, chead), a.D, mild, unused);
                if (MODE != kForward) {
                    bool other;
                    attn_survey<T>(MODE == kGradKV ? attn_at<T>(a, a.q, w.b, at, chead) : attn_at<T>(a, a.k, w.b, at, chead), a.D, other, unused);
                    mild = mild && other;
                }
                if (MODE == kGradKV) {
                    const float *st = attn_stat(a, w.b, chead, at);
                    number = st[0] == st[0];
                    mild = mild && isfinite(st[2]);
                }
            }
            const uint32_t there = __ballot_sync(0xffffffffu, at < len), wild = __ballot_sync(0xffffffffu, !mild), nan = __ballot_sync(0xffffffffu, !number);
            const uint32_t on = attn_word<MODE>(a, words, cpos + c0) & there, off = ~on & there;
            allowed = allowed || on;
            masked = masked || off;
            cause = cause || (off & wild);
            lost = lost || (on & nan) || (MODE == kGradQ && !finite && on);
        }
        if (__all_sync(0xffffffffu, lost)) return false;
    }
    return !lost && (cause || (finite ? !tame && masked : !allowed));
}

// Row r from its allowed pairs alone: by one warp, column by column, slowly. The caller's
// sums have the row's reference maximum `m2` (forward, in the exponent's units). acc1 and
// acc2: channels lane, lane + 32, ... of p x2 and ds x1.
template <typename T, int MODE, int C>
__device__ __noinline__ void attn_exact_row(const AttnArgs &a, const AttnRows &w, int r, int64_t j0, int64_t j1,
                                            float m2, float (&acc1)[4], float (&acc2)[4]) {
    constexpr int V = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const int pos = w.row_pos(r), head = w.row_head(r);
    const T *a1 = MODE == kGradKV ? attn_at<T>(a, a.k, w.b, pos, head) : attn_at<T>(a, a.q, w.b, pos, head);
    const T *a2 = MODE == kGradKV ? attn_at<T>(a, a.v, w.b, pos, head)
                                  : MODE == kGradQ ? attn_at<T>(a, a.go, w.b, pos, head) : nullptr;
    float lse2 = m2, delta = 0.0f;
    if (MODE == kGradQ) {
        const float *st = attn_stat(a, w.b, head, pos);
        lse2 = a.up - st[0];
        delta = -st[2];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc1[i] = acc2[i] = 0.0f;
    for (int64_t j = j0; j < j1; ++j) {
        int cpos, chead;
        attn_columns<MODE, C>(a, w, j, &cpos, &chead);
        if (!attn_class<MODE, C>(a, w, cpos, chead)) continue;
        const uint32_t *words = attn_word_row<MODE>(a, w.b, MODE == kGradKV ? chead : head, pos);
        for (int c0 = 0; c0 < C; c0 += 32) {
            const int at = cpos + c0 + lane, len = MODE == kGradKV ? a.Q : a.S;
            if (cpos + c0 >= len) break;
            bool on = at < len && ((attn_word<MODE>(a, words, cpos + c0) >> lane) & 1u);
            const T *x1 = nullptr, *x2 = nullptr;
            float p = 0.0f, ds = 0.0f;
            if (on) {
                x1 = MODE == kGradKV ? attn_at<T>(a, a.q, w.b, at, chead) : attn_at<T>(a, a.k, w.b, at, chead);
                x2 = MODE == kGradKV ? attn_at<T>(a, a.go, w.b, at, chead) : attn_at<T>(a, a.v, w.b, at, chead);
                float s = 0.0f, dp = 0.0f;
                for (int d = 0; d < a.D; d += V) {
                    float y[V], z[V];
                    unpack16<T>(y, ldg16(a1 + d));
                    unpack16<T>(z, ldg16(x1 + d));
#pragma unroll
                    for (int k = 0; k < V; ++k) s = fmaf(y[k], z[k], s);
                    if (MODE == kForward) continue;
                    unpack16<T>(y, ldg16(a2 + d));
                    unpack16<T>(z, ldg16(x2 + d));
#pragma unroll
                    for (int k = 0; k < V; ++k) dp = fmaf(y[k], z[k], dp);
                }
                if (MODE == kGradKV) {
                    const float *st = attn_stat(a, w.b, chead, at);
                    lse2 = a.up - st[0];
                    delta = -st[2];
                }
                if (MODE != kForward) on = lse2 != INFINITY;
                p = on ? exp2f(fmaf(s, a.c, -lse2)) : 0.0f;
                ds = on ? p * (dp - delta) : 0.0f;
            }
            // four allowed columns at a time, their loads under way together
            const T *rows1 = MODE == kGradKV ? attn_at<T>(a, a.q, w.b, cpos + c0, chead) : attn_at<T>(a, a.k, w.b, cpos + c0, chead);
            const T *rows2 = MODE == kGradKV ? attn_at<T>(a, a.go, w.b, cpos + c0, chead) : attn_at<T>(a, a.v, w.b, cpos + c0, chead);
            const int64_t step1 = MODE == kGradKV ? a.q.pos : a.k.pos, step2 = MODE == kGradKV ? a.go.pos : a.v.pos;
            for (uint32_t left = __ballot_sync(0xffffffffu, on); left;) {
                constexpr int U = 4;
                float pf[U], df[U], y1[U][4], y2[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool any = left != 0u;       // of the whole warp
                    const int from = any ? __ffs(left) - 1 : 0;
                    left &= left - 1;
                    pf[u] = __shfl_sync(0xffffffffu, any ? p : 0.0f, from);
                    df[u] = __shfl_sync(0xffffffffu, any ? ds : 0.0f, from);
                    const T *r1 = rows1 + from * step1 + lane, *r2 = rows2 + from * step2 + lane;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool there = any && lane + 32 * i < a.D;
                        if (MODE != kForward) y1[u][i] = there ? Elem<T>::to_f(r1[32 * i]) : 0.0f;
                        if (MODE != kGradQ) y2[u][i] = there ? Elem<T>::to_f(r2[32 * i]) : 0.0f;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (MODE != kGradQ) acc1[i] = fmaf(pf[u], y2[u][i], acc1[i]);
                        if (MODE != kForward) acc2[i] = fmaf(df[u], y1[u][i], acc2[i]);
                    }
            }
        }
    }
}

// A value of the output, and what its rounding left.
template <typename T> __device__ __forceinline__ void attn_put(const AttnArgs &a, void *out, void *rest, int64_t at, float v) {
    if (!attn_ok(a, at, a.part_rows * a.D)) return;
    const T rounded = Elem<T>::from_f(v);
    static_cast<T *>(out)[at] = rounded;
    if (rest) static_cast<T *>(rest)[at] = Elem<T>::from_f(v - Elem<T>::to_f(rounded));
}

// One result of a row: a value of the output, or of this split's part. which: 0,
// or 1 for the second of a key's gradients; f: what the sum is multiplied by.
template <typename T, int MODE>
__device__ __forceinline__ void attn_store(const AttnArgs &a, const AttnRows &w, int r, int split, int which, int d,
                                           float sum, float f) {
    const int pos = w.row_pos(r), head = w.row_head(r);
    const int len = MODE == kGradKV ? a.S : a.Q, heads = MODE == kGradKV ? a.N : a.M;
    const int64_t row = ((int64_t)w.b * len + pos) * heads + head;
    if (a.splits > 1) {
        a.part[((int64_t)(which * a.splits + split) * a.part_rows + row) * a.D + d] = sum;
        return;
    }
    void *to = MODE == kForward ? a.out : MODE == kGradQ ? a.gq : which ? a.gk : a.gv;
    attn_put<T>(a, to, MODE == kForward ? a.rest : nullptr, row * a.D + d, sum * f);
}

}  // namespace msda
