// Layer norm's C entries: argument validation and the choice of kernel (host
// code; contracts in include/msda.h).
#include "msda_norm.cuh"

namespace msda {
cudaError_t launch_norm_forward(const NormArgs &a, const NormPlan &p, msda_dtype_t dt,
                                msda_dtype_t pdt, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormArgs &a, const NormPlan &p, msda_dtype_t dt,
                                 msda_dtype_t pdt, cudaStream_t stream);
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

// How rows of C elements are held (see msda_norm.cuh). `aligned16`: every
// tensor of rows starts on a 16-byte boundary. Two granules a thread: measured
// against one, two, three and four on rows of 64 to 8192 channels, they were the
// fastest or within 3% (one spends more on the row's sums, four leave too few
// warps); rows past 512 * 2 granules take four.
NormPlan row_plan(const msda_norm_dims_t &d, msda_dtype_t dt, bool aligned16, int threads) {
    NormPlan p = {};
    const int V = 16 / elem_bytes(dt);
    p.ragged = d.C % V != 0;
    // granules of a row, the most that any phase touches
    const int64_t n = p.ragged ? (d.C + V - 1 + V - 1) / V : d.C / V;
    p.KV = n <= 1024 ? 2 : 4;
    if (dt == MSDA_F64 || !aligned16 || n > 2048) {
        p.general = true;
        return p;
    }
    if (n <= 64) {
        p.G = n <= 4 ? 2 : n <= 8 ? 4 : n <= 16 ? 8 : n <= 32 ? 16 : 32;
        p.group = p.G;
        p.threads = threads;
    } else {
        p.group = (int)((n + p.KV - 1) / p.KV + 31) / 32 * 32;
        p.threads = p.group >= threads ? p.group : threads / p.group * p.group;
    }
    return p;
}

NormPlan forward_plan(const msda_norm_dims_t &d, msda_dtype_t dt, bool aligned16) {
    NormPlan p = row_plan(d, dt, aligned16, msda::kForwardThreads);
    if (p.general) {
        p.threads = 512;
        p.blocks = (int)(d.N < (1 << 30) ? d.N : (1 << 30));
        return p;
    }
    const int64_t per_block = p.threads / p.group, want = (d.N + per_block - 1) / per_block;
    const int64_t cap = msda::kSMs * (1024 / p.threads);
    p.blocks = (int)(want < cap ? want : cap);
    return p;
}

// The backward's blocks walk many rows each, since each leaves a row of
// partial column sums (general: the count of row chunks).
NormPlan backward_plan(const msda_norm_dims_t &d, msda_dtype_t dt, bool aligned16) {
    NormPlan p = row_plan(d, dt, aligned16, msda::kBackwardThreads);
    if (p.general) {
        p.threads = 512;
        p.blocks = (int)(d.N < 1 ? 1 : d.N < 256 ? d.N : 256);
        return p;
    }
    const int64_t per_block = p.threads / p.group, want = (d.N + per_block - 1) / per_block;
    const int64_t cap = msda::kSMs * (p.threads > 256 ? 1 : 512 / p.threads);
    p.blocks = (int)(want < 1 ? 1 : want < cap ? want : cap);
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
    return from_cuda(msda::launch_norm_forward(a, p, dtype, param_dtype,
                                               static_cast<cudaStream_t>(stream)));
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
    a.N = d.N;
    a.C = (int)d.C;
    a.group = p.group;
    return from_cuda(msda::launch_norm_backward(a, p, dtype, param_dtype,
                                                static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
