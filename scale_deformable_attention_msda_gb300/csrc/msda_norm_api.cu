// Layer norm's C entries: argument validation and the choice of kernel (host
// code; contracts in include/msda.h).
#include "msda_norm.cuh"

namespace msda {
cudaError_t launch_norm_forward_f32(const NormArgs &a, const NormPlan &p, cudaStream_t stream);
cudaError_t launch_norm_forward_f64(const NormArgs &a, const NormPlan &p, cudaStream_t stream);
cudaError_t launch_norm_forward_bf16(const NormArgs &a, const NormPlan &p, bool wide, cudaStream_t stream);
cudaError_t launch_norm_forward_f16(const NormArgs &a, const NormPlan &p, bool wide, cudaStream_t stream);
cudaError_t launch_norm_backward_f32(const NormArgs &a, const NormPlan &p, cudaStream_t stream);
cudaError_t launch_norm_backward_f64(const NormArgs &a, const NormPlan &p, cudaStream_t stream);
cudaError_t launch_norm_backward_bf16(const NormArgs &a, const NormPlan &p, bool wide, cudaStream_t stream);
cudaError_t launch_norm_backward_f16(const NormArgs &a, const NormPlan &p, bool wide, cudaStream_t stream);
cudaError_t fault_word_for_launch(unsigned **err);
}  // namespace msda

namespace {

using msda::NormArgs;
using msda::NormPlan;

constexpr int64_t kMaxColumns = 1 << 20;
constexpr int64_t kMaxElements = (int64_t)1 << 60;

int elem_bytes(msda_dtype_t dt) { return dt == MSDA_F64 ? 8 : (dt == MSDA_F32 ? 4 : 2); }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

msda_status_t check(const msda_norm_dims_t *d, msda_dtype_t dt, msda_dtype_t pdt) {
    if (!d) return MSDA_ERR_NULL;
    if (dt != MSDA_F32 && dt != MSDA_BF16 && dt != MSDA_F16 && dt != MSDA_F64) return MSDA_ERR_DTYPE;
    if (pdt != dt && !(pdt == MSDA_F32 && (dt == MSDA_BF16 || dt == MSDA_F16))) return MSDA_ERR_DTYPE;
    if (d->N < 0 || d->C < 1 || d->C > kMaxColumns || d->N > kMaxElements / d->C) return MSDA_ERR_SHAPE;
    return MSDA_OK;
}

// The longest rows of the tiles form. Forward: 32 channels for each of 512
// threads, two tensors and two results in a block's shared memory. Backward: 16
// channels; with 32 its sums leave the registers, and 1,249 rows of 12,001 bf16
// take 127 us against the general form's 94.
constexpr int64_t max_tile_columns(msda_dtype_t dt, bool backward) {
    return backward ? 512 * msda::kTileE : dt == MSDA_F32 ? (int64_t)(msda::kMostShared / (4 * 4)) - 16 : 16384;
}

// Threads of a group of whole warps with room for `items` at `per` each.
int warps_for(int64_t items, int per) { return (int)((items + per - 1) / per + 31) / 32 * 32; }

// The rows form for rows of n granules, as measured on rows of 64 to 8192
// channels at each of 2, 3 and 4 granules a thread. Fewer lanes a row spend less
// on its sums, and idle lanes cost more than that. Lanes of a warp, up to 128
// granules: two granules a thread, three where that leaves fewer lanes idle, four
// past 96 (14,600 x 1024 bf16 forward: 12.2 us, two 15.0; 15,600 x 512 fp32
// backward 19.7 us, two 21.9). The 16-bit backward, with twice the channels in a
// granule and sums beside them, stays with two (14,600 x 1024: 21.8 us, four
// 25.1), but for three just past 64 granules (23,000 x 640: 26.1 us, two 27.5).
// Groups of warps: four granules, but two of the 16-bit backward's and of 16-bit
// rows that would leave more than a tenth of the lanes idle (5,990 x 2504 forward:
// 16.8 us, four 19.4; 3,000 x 5000: 18.1 us, four 14.7), while they hold the row.
void hold_rows(int64_t n, bool narrow, bool backward, NormPlan *p) {
    p->form = NormPlan::kRows;
    int g = 2;
    while (2 * g < n && g < 32) g *= 2;
    const bool two = narrow && backward;
    if (n <= (two ? 80 : 128)) {
        p->KV = n <= 2 * g ? 2 : n <= 3 * g ? 3 : 4;
        if (!two && p->KV == 2 && g > 2 && 2 * n <= 3 * g) {
            g /= 2;
            p->KV = 3;
        }
        p->G = p->group = g;
        p->threads = msda::kGroupThreads;
    } else {
        const bool idle = 10 * n < 9 * 4 * warps_for(n, 4);
        p->KV = narrow && n <= 1024 && (backward || idle) ? 2 : n <= 2048 ? 4 : 8;
        p->G = 0;
        p->group = warps_for(n, p->KV);
        p->threads = p->group >= 256 ? p->group : 256 / p->group * p->group;
    }
}

// The tiles form: the fewest threads with at most 16 channels each (32 in the
// longest rows); more than 8 each but for the shortest.
void hold_tiles(int64_t C, NormPlan *p) {
    p->form = NormPlan::kTiles;
    const int64_t t = (C + msda::kTileE - 1) / msda::kTileE;
    if (t <= 32) {
        int g = 2;
        while (g < t) g *= 2;
        p->G = p->group = g;
        p->threads = msda::kTileThreads;
    } else {
        p->G = 0;
        p->group = t < 512 ? warps_for(C, msda::kTileE) : 512;
        p->threads = p->group >= msda::kTileThreads ? p->group : msda::kTileThreads / p->group * p->group;
    }
    p->KV = C <= 8 * p->group ? 4 : C <= 12 * p->group ? 6 : C <= 16 * p->group ? 8 : 16;
}

// `aligned16`: every tensor of rows starts on a 16-byte boundary.
NormPlan row_plan(const msda_norm_dims_t &d, msda_dtype_t dt, bool aligned16, bool backward) {
    NormPlan p = {};
    const int V = 16 / elem_bytes(dt);
    // no rows: the general form touches nothing of the tensors of rows
    const bool general = dt == MSDA_F64 || d.N == 0;
    // eight granules of fp32 are four of 16 bits; the backward's 416 threads are
    // what the copies of four tensors leave of a block's shared memory
    const int64_t most = dt != MSDA_F32 ? 2048 : backward ? 8 * 416 : 8 * 512;
    if (!general && d.C % V == 0 && aligned16 && d.C / V <= most) {
        hold_rows(d.C / V, dt != MSDA_F32, backward, &p);
    } else if (!general && d.C <= max_tile_columns(dt, backward)) {
        hold_tiles(d.C, &p);
    } else {
        p.form = NormPlan::kGeneral;
        p.group = p.threads = 512;
    }
    return p;
}

// Blocks for `per_sm` threads on each SM, or as many as there are rows for.
int blocks_of(const msda_norm_dims_t &d, const NormPlan &p, int per_sm) {
    const int64_t per_block = p.threads / p.group, want = (d.N + per_block - 1) / per_block;
    const int64_t cap = msda::kSMs * (per_sm > p.threads ? per_sm / p.threads : 1);
    return (int)(want < 1 ? 1 : want < cap ? want : cap);
}

// Where a thread has three or four granules of two rows under way, 512 threads of
// an SM are enough; more of them share fewer rows each, and pay for their start.
NormPlan forward_plan(const msda_norm_dims_t &d, msda_dtype_t dt, bool aligned16) {
    NormPlan p = row_plan(d, dt, aligned16, false);
    if (p.form == NormPlan::kGeneral) p.blocks = (int)(d.N < (1 << 30) ? d.N : (1 << 30));
    else p.blocks = blocks_of(d, p, p.form == NormPlan::kRows && p.G > 0 && p.KV > 2 ? 512 : 1024);
    return p;
}

// The backward's blocks walk many rows each, since each leaves a row of
// partial column sums (general: the count of row chunks).
NormPlan backward_plan(const msda_norm_dims_t &d, msda_dtype_t dt, bool aligned16) {
    NormPlan p = row_plan(d, dt, aligned16, true);
    if (p.form == NormPlan::kGeneral) p.blocks = (int)(d.N < 1 ? 1 : d.N < 256 ? d.N : 256);
    else p.blocks = blocks_of(d, p, 512);
    return p;
}

// The most blocks any plan of these sizes takes: which one depends on the
// pointers' alignment, which the size query does not see.
size_t backward_bytes(const msda_norm_dims_t &d, msda_dtype_t dt) {
    const int a = backward_plan(d, dt, true).blocks, b = backward_plan(d, dt, false).blocks;
    return (size_t)(a > b ? a : b) * 2 * (size_t)d.C * (dt == MSDA_F64 ? 8 : 4);
}

bool aligned16(const void *const *p, int count) {
    for (int i = 0; i < count; ++i)
        if (!aligned(p[i], 16)) return false;
    return true;
}

// Launches of a type checked before.
cudaError_t launch_forward(const NormArgs &a, const NormPlan &p, msda_dtype_t dt, msda_dtype_t pdt,
                           cudaStream_t stream) {
    const bool wide = pdt == MSDA_F32;
    switch (dt) {
        case MSDA_F32: return msda::launch_norm_forward_f32(a, p, stream);
        case MSDA_F64: return msda::launch_norm_forward_f64(a, p, stream);
        case MSDA_BF16: return msda::launch_norm_forward_bf16(a, p, wide, stream);
        default: return msda::launch_norm_forward_f16(a, p, wide, stream);
    }
}
cudaError_t launch_backward(const NormArgs &a, const NormPlan &p, msda_dtype_t dt, msda_dtype_t pdt,
                            cudaStream_t stream) {
    const bool wide = pdt == MSDA_F32;
    switch (dt) {
        case MSDA_F32: return msda::launch_norm_backward_f32(a, p, stream);
        case MSDA_F64: return msda::launch_norm_backward_f64(a, p, stream);
        case MSDA_BF16: return msda::launch_norm_backward_bf16(a, p, wide, stream);
        default: return msda::launch_norm_backward_f16(a, p, wide, stream);
    }
}

msda_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MSDA_OK : MSDA_ERR_CUDA; }

}  // namespace

extern "C" {

msda_status_t msda_layer_norm_forward(const void *x, const void *residual, const void *weight,
                                      const void *bias, void *out, void *sum, void *mean,
                                      void *rstd, double eps, const msda_norm_dims_t *dims,
                                      msda_dtype_t dtype, msda_dtype_t param_dtype, void *stream) {
    const msda_status_t st = check(dims, dtype, param_dtype);
    if (st != MSDA_OK) return st;
    if (!(eps >= 0.0)) return MSDA_ERR_SHAPE;
    const msda_norm_dims_t &d = *dims;
    if (d.N == 0) return MSDA_OK;
    if (!x || !out || (mean == nullptr) != (rstd == nullptr)) return MSDA_ERR_NULL;
    const int e = elem_bytes(dtype), pe = elem_bytes(param_dtype), se = dtype == MSDA_F64 ? 8 : 4;
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(out, e) || !aligned(sum, e) ||
        !aligned(weight, pe) || !aligned(bias, pe) || !aligned(mean, se) || !aligned(rstd, se))
        return MSDA_ERR_ALIGN;
    const void *const all[] = {x, residual, out, sum, weight, bias};
    const NormPlan p = forward_plan(d, dtype, aligned16(all, 6));
    NormArgs a = {};
    if (msda::fault_word_for_launch(&a.err) != cudaSuccess) return MSDA_ERR_CUDA;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.bias = bias;
    a.out = out;
    a.sum = sum;
    a.mean = mean;
    a.rstd = rstd;
    a.eps = eps;
    a.N = d.N;
    a.C = (int)d.C;
    a.group = p.group;
    return from_cuda(launch_forward(a, p, dtype, param_dtype, static_cast<cudaStream_t>(stream)));
}

size_t msda_layer_norm_backward_workspace_bytes(const msda_norm_dims_t *dims, msda_dtype_t dtype) {
    if (check(dims, dtype, dtype) != MSDA_OK) return 0;
    return backward_bytes(*dims, dtype);
}

msda_status_t msda_layer_norm_backward(const void *grad_out, const void *grad_sum, const void *x,
                                       const void *residual, const void *weight,
                                       const void *mean, const void *rstd, void *grad_x,
                                       void *grad_weight, void *grad_bias, void *workspace,
                                       size_t workspace_bytes, const msda_norm_dims_t *dims,
                                       msda_dtype_t dtype, msda_dtype_t param_dtype, void *stream) {
    const msda_status_t st = check(dims, dtype, param_dtype);
    if (st != MSDA_OK) return st;
    const msda_norm_dims_t &d = *dims;
    const bool columns = grad_weight || grad_bias;
    if (!grad_x && !columns) return MSDA_OK;
    if (d.N > 0 && (!grad_out || !x || !mean || !rstd)) return MSDA_ERR_NULL;
    const int e = elem_bytes(dtype), pe = elem_bytes(param_dtype), se = dtype == MSDA_F64 ? 8 : 4;
    if (!aligned(grad_out, e) || !aligned(grad_sum, e) || !aligned(x, e) || !aligned(residual, e) ||
        !aligned(grad_x, e) || !aligned(weight, pe) || !aligned(grad_weight, pe) ||
        !aligned(grad_bias, pe) || !aligned(mean, se) || !aligned(rstd, se))
        return MSDA_ERR_ALIGN;
    if (columns && (!workspace || workspace_bytes < backward_bytes(d, dtype)))
        return MSDA_ERR_WORKSPACE;
    if (columns && !aligned(workspace, 16)) return MSDA_ERR_ALIGN;
    if (d.N == 0 && !columns) return MSDA_OK;   // N = 0 with columns: they are written as zeros
    const void *const all[] = {grad_out, grad_sum, x, residual, weight, grad_x};
    const NormPlan p = backward_plan(d, dtype, aligned16(all, 6));
    NormArgs a = {};
    if (msda::fault_word_for_launch(&a.err) != cudaSuccess) return MSDA_ERR_CUDA;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.mean = const_cast<void *>(mean);
    a.rstd = const_cast<void *>(rstd);
    a.grad_out = grad_out;
    a.grad_sum = grad_sum;
    a.grad_x = d.N > 0 ? grad_x : nullptr;
    a.grad_weight = grad_weight;
    a.grad_bias = grad_bias;
    a.partial = columns ? static_cast<float *>(workspace) : nullptr;
    a.partials = (int64_t)(workspace_bytes / (dtype == MSDA_F64 ? 8 : 4));
    a.N = d.N;
    a.C = (int)d.C;
    a.group = p.group;
    return from_cuda(launch_backward(a, p, dtype, param_dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
