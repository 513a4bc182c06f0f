// Attention's C entries: argument validation, the workspace's layout and the
// order of launches (host code; contracts in include/msda.h).
#include <math.h>

#include "msda_attention_host.h"
#include "msda_host.h"

namespace {

using msda::AttnArgs;
using msda::AttnMode;

constexpr int kSMs = 152;
constexpr int64_t kMaxPositions = (int64_t)1 << 30, kMaxHeads = 65536, kMaxStride = (int64_t)1 << 36;
constexpr int64_t kMaxTiles = ((int64_t)1 << 31) - 1;
constexpr int kDeltaBlocks = 608;

int elem_bytes(msda_dtype_t dt) { return dt == MSDA_F32 ? 4 : 2; }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool stride_ok(int64_t stride, int64_t length, int e) {
    return length <= 1 || (stride > 0 && stride < kMaxStride && stride * e % 16 == 0);
}

msda_status_t check(const msda_attention_dims_t *d, msda_dtype_t dt, bool mask) {
    if (!d) return MSDA_ERR_NULL;
    if (dt != MSDA_F32 && dt != MSDA_BF16 && dt != MSDA_F16) return MSDA_ERR_DTYPE;
    if (d->B < 0 || d->Q < 0 || d->S < 0 || d->Q > kMaxPositions || d->S > kMaxPositions) return MSDA_ERR_SHAPE;
    if (d->N < 1 || d->M < d->N || d->M > kMaxHeads || d->M % d->N) return MSDA_ERR_SHAPE;
    if (d->D < 8 || d->D > msda::kAttnMaxD || d->D % 8) return MSDA_ERR_SHAPE;
    const int64_t longest = d->Q > d->S ? d->Q : d->S;
    if (d->B > 0 && d->B > kMaxTiles / d->M / (longest / 64 + 1)) return MSDA_ERR_SHAPE;
    if (mask && d->B > 0 && ceil_div(d->Q, 64) * ceil_div(d->S, 128) > kMaxTiles / (d->B * d->M)) return MSDA_ERR_SHAPE;
    const int e = elem_bytes(dt);
    const int64_t len[3] = {d->B, 0, 0};
    const int64_t *strides[3] = {d->q_stride, d->k_stride, d->v_stride};
    for (int t = 0; t < 3; ++t) {
        const int64_t size[3] = {len[0], t ? d->S : d->Q, t ? d->N : d->M};
        if (size[0] * size[1] == 0) continue;                  // nothing there
        for (int i = 0; i < 3; ++i)
            if (!stride_ok(strides[t][i], size[i], e))
                return strides[t][i] > 0 && strides[t][i] < kMaxStride ? MSDA_ERR_ALIGN : MSDA_ERR_SHAPE;
    }
    if (mask)
        for (int i = 0; i < 4; ++i)
            if (d->mask_stride[i] < 0 || d->mask_stride[i] > ((int64_t)1 << 60)) return MSDA_ERR_SHAPE;
    return MSDA_OK;
}

// Query heads in one row tile: all that share a key head where the queries alone
// do not fill it.
int pack_of(const msda_attention_dims_t &d, int rows) {
    const int64_t g = d.M / d.N;
    return g > 1 && g <= rows && d.Q < rows ? (int)g : 1;
}

struct ModePlan {
    int64_t tiles, blocks;             // row tiles; blocks = tiles * splits
    int splits;
    size_t part;                       // bytes of the splits' results
};

// Splits of a row tile's columns: as many as fill the SMs, but none of fewer than
// `least` column tiles.
ModePlan plan_mode(const msda_attention_dims_t &d, AttnMode mode, int R, int C, int slots, int least) {
    ModePlan p = {};
    const int64_t len = mode == msda::kGradKV ? d.S : d.Q;
    const int pack = mode == msda::kGradKV ? 1 : pack_of(d, R);
    const int64_t heads = mode == msda::kGradKV ? d.N : d.M / pack;
    p.tiles = d.B * heads * ceil_div(len, R / pack);
    const int64_t columns = mode == msda::kGradKV ? d.M / d.N * ceil_div(d.Q, C) : ceil_div(d.S, C);
    int64_t s = p.tiles > 0 ? slots / p.tiles : 1;
    if (s > columns / least) s = columns / least;
    if (s > 64) s = 64;
    p.splits = (int)(s < 1 ? 1 : s);
    p.blocks = p.tiles * p.splits;
    if (p.splits > 1) {
        const int64_t rows = d.B * len * (mode == msda::kGradKV ? d.N : d.M);
        p.part = (size_t)p.splits * rows * (d.D * (mode == msda::kGradKV ? 2 : 1) + (mode == msda::kForward ? 2 : 0)) * 4;
    }
    return p;
}

// Blocks of the pass over the queries' rows: one for 64 rows, of which its 256 threads have 32
// to 256 under way at once, and four an SM at most. One for each 8 to 64 rows instead, as many
// as there are threads for: the backward of 600 rows of 4 heads of 128 in fp32 150 us (153),
// of 2 x 300 of 8 heads of 64 in fp16 15.9 (14.5), of 4 x 512 in bf16 24.5 (22.9).
int64_t delta_blocks(int64_t rows) {
    const int64_t blocks = ceil_div(rows, 64);
    return blocks < 1 ? 1 : blocks < kDeltaBlocks ? blocks : kDeltaBlocks;
}
// fp16: parts of a batch entry's and key head's rows, of queries and of keys, in that pass.
int norm_parts(const msda_attention_dims_t &d) {
    const int64_t queries = ceil_div(d.Q, 128) * 128 * (d.M / d.N), most = kDeltaBlocks / 2 / (d.B * d.N);
    const int64_t parts = delta_blocks(queries > d.S ? queries : d.S);
    return (int)(most < 1 ? 1 : parts < most ? parts : most);
}

int tile_rows(msda_dtype_t dt) { return dt == MSDA_F32 ? 64 : 128; }

ModePlan plan_for(const msda_attention_dims_t &d, msda_dtype_t dt, AttnMode mode) {
    if (msda::few_rows(mode, dt, d.Q, d.M / d.N)) {
        // a key head's keys over as many blocks as two an SM leave it, 256 keys or more for each
        // (their shares are rounded up to 32 keys, and the last one has what is left)
        ModePlan p = {};
        p.tiles = d.B * d.N;
        int64_t s = p.tiles > 0 ? 2 * kSMs / p.tiles : 1;
        if (s > d.S / 256) s = d.S / 256;
        p.splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
        p.blocks = p.tiles * p.splits;
        if (p.splits > 1) p.part = (size_t)p.splits * d.B * d.Q * d.M * (d.D + 2) * 4;
        return p;
    }
    if (dt == MSDA_F32) return plan_mode(d, mode, 64, 64, kSMs * msda::simple_blocks(d.D), 1);
    const bool is_short = msda::tc_short(mode, d.D, d.Q, d.M / d.N, d.B * d.N * ceil_div(d.S, 128));
    const int columns = msda::tc_columns(mode, d.D, is_short), blocks = msda::tc_blocks(mode, d.D, is_short);
    return plan_mode(d, mode, 128, columns, kSMs * blocks, 4);
}

// The workspace, each piece on a 256-byte boundary.
struct Layout {
    size_t bits_q, bits_k, classes, stat, norms, part[3], bytes;
    int mb, mm, mq, words_q, words_k, granules;    // the mask's own extents (1 where it repeats)
};

Layout layout_of(const msda_attention_dims_t &d, msda_dtype_t dt, bool mask, bool backward) {
    Layout w = {};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    if (mask) {
        // a mask that repeats along a dimension is packed once for all of it
        w.mb = d.B > 1 && d.mask_stride[0] == 0 ? 1 : (int)d.B;
        w.mm = d.mask_stride[1] == 0 ? 1 : (int)d.M;
        w.mq = d.mask_stride[2] == 0 ? 1 : (int)d.Q;
        w.granules = (int)(2 * ceil_div(d.S, 128));
        w.words_q = 2 * w.granules;
        w.words_k = w.mq > 1 ? (int)(2 * ceil_div(w.mq, 64)) : 1;
        const size_t maps = (size_t)w.mb * w.mm;
        w.bits_q = take(maps * w.mq * w.words_q * 4);
        w.classes = take(maps * ceil_div(w.mq, 64) * w.granules);
        if (backward) w.bits_k = take(maps * d.S * w.words_k * 4);
    }
    if (backward) {
        w.stat = take((size_t)d.B * d.M * ceil_div(d.Q, 128) * 128 * 8);
        if (dt == MSDA_F16 && d.B > 0) w.norms = take((size_t)2 * d.B * d.N * norm_parts(d) * 4);
        w.part[1] = take(plan_for(d, dt, msda::kGradQ).part);
        w.part[2] = take(plan_for(d, dt, msda::kGradKV).part);
    } else {
        w.part[0] = take(plan_for(d, dt, msda::kForward).part);
    }
    w.bytes = at;
    return w;
}

msda::AttnTensor strided(const void *p, const int64_t *s, int64_t len, int64_t heads) { return {p, s[0], s[1], s[2], (int)len, (int)heads}; }
msda::AttnTensor dense(const void *p, int64_t len, int64_t heads, int64_t D) {
    return {p, len * heads * D, heads * D, D, (int)len, (int)heads};
}

AttnArgs common_args(const msda_attention_dims_t &d, const void *q, const void *k, const void *v, double scale) {
    AttnArgs a = {};
    a.q = strided(q, d.q_stride, d.Q, d.M);
    a.k = strided(k, d.k_stride, d.S, d.N);
    a.v = strided(v, d.v_stride, d.S, d.N);
    a.B = (int)d.B;
    a.Q = (int)d.Q;
    a.S = (int)d.S;
    a.M = (int)d.M;
    a.N = (int)d.N;
    a.D = (int)d.D;
    a.G = (int)(d.M / d.N);
    a.scale = (float)scale;
    // above zero, so that a masked score, -infinity, stays so, and lse / c in range
    a.c = (float)(scale * 1.4426950408889634 > 1e-30 ? scale * 1.4426950408889634 : 1e-30);
    return a;
}

// Packs the mask into the workspace and points the arguments to it.
cudaError_t pack_mask(AttnArgs &a, const msda_attention_dims_t &d, const Layout &w, const void *mask, char *ws,
                      bool backward, cudaStream_t stream) {
    const msda::AttnMaskSource m = {static_cast<const uint8_t *>(mask), d.mask_stride[0], d.mask_stride[1],
                                    d.mask_stride[2], d.mask_stride[3], w.mb, w.mm, w.mq, (int)d.S};
    uint32_t *by_query = reinterpret_cast<uint32_t *>(ws + w.bits_q);
    uint32_t *by_key = backward ? reinterpret_cast<uint32_t *>(ws + w.bits_k) : nullptr;
    uint8_t *classes = reinterpret_cast<uint8_t *>(ws + w.classes);
    const int64_t rows = ceil_div(w.mq, 64);
    const bool heads = w.mm > 1, batches = w.mb > 1;
    a.by_query = {by_query, batches ? (int64_t)w.mm * w.mq * w.words_q : 0, heads ? (int64_t)w.mq * w.words_q : 0,
                  w.mq > 1 ? w.words_q : 0, 1};
    a.by_key = {by_key, batches ? (int64_t)w.mm * d.S * w.words_k : 0, heads ? d.S * w.words_k : 0, w.words_k, w.mq > 1};
    a.classes = classes;
    a.class_batch = batches ? (int64_t)w.mm * rows * w.granules : 0;
    a.class_head = heads ? rows * w.granules : 0;
    a.class_row = w.mq > 1 ? w.granules : 0;
    return msda::launch_attention_pack(m, by_query, w.words_q, by_key, w.words_k, classes, w.granules, stream);
}

// One mode's share of a call: its arguments and blocks.
struct Part {
    AttnMode mode;
    AttnArgs a;
    int64_t blocks;
};
Part part_of(AttnArgs a, const msda_attention_dims_t &d, msda_dtype_t dt, AttnMode mode, char *part) {
    const ModePlan p = plan_for(d, dt, mode);
    a.pack = mode == msda::kGradKV ? 1 : pack_of(d, tile_rows(dt));
    a.splits = p.splits;
    a.part = reinterpret_cast<float *>(part);
    a.part_rows = mode == msda::kGradKV ? d.B * d.S * d.N : d.B * d.Q * d.M;
    return {mode, a, p.blocks};
}
cudaError_t join(const Part &p, msda_dtype_t dt, cudaStream_t stream) {
    return p.blocks > 0 && p.a.splits > 1 ? msda::launch_attention_join(p.mode, p.a, dt, stream) : cudaSuccess;
}

cudaError_t launch_forward(const Part &p, msda_dtype_t dt, cudaStream_t stream) {
    const cudaError_t e = msda::few_rows(p.mode, dt, p.a.Q, p.a.G) ? msda::launch_attention_few(p.a, p.blocks, stream)
                        : dt == MSDA_F32  ? msda::launch_attention_f32(p.mode, p.a, p.blocks, stream)
                        : dt == MSDA_BF16 ? msda::launch_attention_bf16(p.a, p.blocks, stream)
                                          : msda::launch_attention_f16(p.a, p.blocks, stream);
    return e == cudaSuccess ? join(p, dt, stream) : e;
}
// The gradients of the queries, and of keys and values; no blocks: not wanted.
cudaError_t launch_backward(const Part &q, const Part &kv, msda_dtype_t dt, cudaStream_t stream) {
    auto back = [&](const Part &p, const Part &r) {      // 16-bit
        return dt == MSDA_BF16 ? msda::launch_attention_bf16_back(p.a, p.blocks, r.a, r.blocks, stream)
                               : msda::launch_attention_f16_back(p.a, p.blocks, r.a, r.blocks, stream);
    };
    auto one = [&](const Part &p) {
        if (p.blocks == 0) return cudaSuccess;
        Part none = p;
        none.blocks = 0;
        return dt == MSDA_F32 ? msda::launch_attention_f32(p.mode, p.a, p.blocks, stream)
             : p.mode == msda::kGradQ ? back(p, none) : back(none, p);
    };
    // two launches also where one grid would not hold both
    const bool apart = dt == MSDA_F32 || q.blocks == 0 || kv.blocks == 0 || q.blocks + kv.blocks > kMaxTiles ||
                       msda::tc_short(kv.a);
    cudaError_t e = apart ? one(q) : back(q, kv);
    if (e == cudaSuccess) e = join(q, dt, stream);
    if (e == cudaSuccess && apart) e = one(kv);
    return e == cudaSuccess ? join(kv, dt, stream) : e;
}

msda_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MSDA_OK : MSDA_ERR_CUDA; }
// times log2(e) an fp32 number
bool scale_ok(double s) { return s >= 0.0 && s <= 2.3e38; }

}  // namespace

extern "C" {

size_t msda_attention_forward_workspace_bytes(const msda_attention_dims_t *dims, msda_dtype_t dtype, int with_mask) {
    if (check(dims, dtype, with_mask != 0) != MSDA_OK) return 0;
    return layout_of(*dims, dtype, with_mask != 0, false).bytes;
}

size_t msda_attention_backward_workspace_bytes(const msda_attention_dims_t *dims, msda_dtype_t dtype, int with_mask) {
    if (check(dims, dtype, with_mask != 0) != MSDA_OK) return 0;
    return layout_of(*dims, dtype, with_mask != 0, true).bytes;
}

msda_status_t msda_attention_forward(const void *q, const void *k, const void *v, const void *mask, void *out,
                                     void *rest, void *lse, double scale, void *workspace, size_t workspace_bytes,
                                     const msda_attention_dims_t *dims, msda_dtype_t dtype, void *stream) {
    const msda_status_t st = check(dims, dtype, mask != nullptr);
    if (st != MSDA_OK) return st;
    if (!scale_ok(scale)) return MSDA_ERR_SHAPE;
    const msda_attention_dims_t &d = *dims;
    if (d.B == 0 || d.Q == 0) return MSDA_OK;
    if (!q || !out || (d.S > 0 && (!k || !v))) return MSDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(rest, 16) ||
        !aligned(lse, 4))
        return MSDA_ERR_ALIGN;
    const bool masked = mask && d.S > 0;
    const Layout w = layout_of(d, dtype, masked, false);
    if (w.bytes && (!workspace || workspace_bytes < w.bytes)) return MSDA_ERR_WORKSPACE;
    if (w.bytes && !aligned(workspace, 16)) return MSDA_ERR_ALIGN;
    AttnArgs a = common_args(d, q, k, v, scale);
    a.out = out;
    a.rest = rest;
    a.lse = static_cast<float *>(lse);
    if (msda::fault_word(&a.err) != cudaSuccess) return MSDA_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = masked ? pack_mask(a, d, w, mask, ws, false, s) : cudaSuccess;
    a.chained = masked;
    if (e == cudaSuccess) e = launch_forward(part_of(a, d, dtype, msda::kForward, ws + w.part[0]), dtype, s);
    return from_cuda(e);
}

msda_status_t msda_attention_backward(const void *grad_out, const void *q, const void *k, const void *v,
                                      const void *mask, const void *out, const void *rest, const void *lse,
                                      void *grad_q, void *grad_k, void *grad_v, double scale, void *workspace, size_t workspace_bytes,
                                      const msda_attention_dims_t *dims, msda_dtype_t dtype, void *stream) {
    const msda_status_t st = check(dims, dtype, mask != nullptr);
    if (st != MSDA_OK) return st;
    if (!scale_ok(scale)) return MSDA_ERR_SHAPE;
    const msda_attention_dims_t &d = *dims;
    if ((grad_k == nullptr) != (grad_v == nullptr)) return MSDA_ERR_NULL;
    const bool for_q = grad_q && d.B * d.Q > 0, for_kv = grad_k && d.B * d.S > 0;
    if (!for_q && !for_kv) return MSDA_OK;
    if (d.Q > 0 && (!grad_out || !q || !out || !lse)) return MSDA_ERR_NULL;
    if (d.S > 0 && (!k || !v)) return MSDA_ERR_NULL;
    if (!aligned(grad_out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned(rest, 16) || !aligned(lse, 4) || !aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(grad_v, 16))
        return MSDA_ERR_ALIGN;
    const bool masked = mask && d.S > 0 && d.Q > 0;
    const Layout w = layout_of(d, dtype, masked, true);
    if (w.bytes && (!workspace || workspace_bytes < w.bytes)) return MSDA_ERR_WORKSPACE;
    if (w.bytes && !aligned(workspace, 16)) return MSDA_ERR_ALIGN;
    AttnArgs a = common_args(d, q, k, v, scale);
    a.go = dense(grad_out, d.Q, d.M, d.D);
    a.o = dense(out, d.Q, d.M, d.D);
    a.lse = static_cast<float *>(const_cast<void *>(lse));
    a.rest = const_cast<void *>(rest);
    a.gq = grad_q;
    a.gk = grad_k;
    a.gv = grad_v;
    if (msda::fault_word(&a.err) != cudaSuccess) return MSDA_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.stat = reinterpret_cast<float *>(ws + w.stat);
    a.stat_row = (int)(ceil_div(d.Q, 128) * 128);
    a.up = dtype == MSDA_F16 ? msda::kHalfUp : 0.0f;
    int64_t blocks = delta_blocks(d.B * a.stat_row * d.M);
    if (dtype == MSDA_F16) {
        a.norms = norm_parts(d);
        a.norm_do = reinterpret_cast<float *>(ws + w.norms);
        a.norm_v = a.norm_do + d.B * d.N * a.norms;
        blocks = 2 * d.B * d.N * a.norms < kDeltaBlocks ? 2 * d.B * d.N * a.norms : kDeltaBlocks;
    }
    cudaError_t e = masked ? pack_mask(a, d, w, mask, ws, true, s) : cudaSuccess;
    a.chained = masked;
    if (e == cudaSuccess) e = msda::launch_attention_delta(a, blocks, dtype, s);
    a.chained = true;
    Part pq = part_of(a, d, dtype, msda::kGradQ, ws + w.part[1]), pkv = part_of(a, d, dtype, msda::kGradKV, ws + w.part[2]);
    if (!for_q) pq.blocks = 0;
    if (!for_kv) pkv.blocks = 0;
    if (e == cudaSuccess) e = launch_backward(pq, pkv, dtype, s);
    return from_cuda(e);
}

}  // extern "C"
