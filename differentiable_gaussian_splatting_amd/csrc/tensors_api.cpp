// tensors_api.cpp -- the C ABI of the table, tensor-list and layer calls
// (declared in include/gs.h): argument checks, workspaces and launches.
#include <cmath>

#include "gs_internal.h"

namespace {

constexpr int64_t kMaxIndex = (1ll << 31) - 1;

size_t type_size(int type) { return type == GS_F32 ? 4 : 2; }

// A descriptor that a kernel may follow: a known type, sizes whose offsets fit
// 64 bits, rows that do not overlap where they are written, and an aligned
// pointer wherever there is a value.
gs_status check_tensor(gs_ctx* ctx, const gs_tensor* t, bool written, const char* what, int32_t k = 0)
{
    if (!t) return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s is NULL", what);
    if (t->type != GS_F32 && t->type != GS_F16 && t->type != GS_BF16)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d: element type %d", what, k, t->type);
    if (t->rows < 0 || t->cols < 0 || t->stride < 0)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d: negative size or stride", what, k);
    if (t->rows == 0 || t->cols == 0) return GS_OK;
    if (t->rows > (1ll << 40) / t->cols || t->cols > (1ll << 40) ||
        (t->stride > 0 && t->rows > (1ll << 60) / t->stride))
        return gs_fail(ctx, GS_ERR_OVERFLOW, "%s %d: %lld x %lld values", what, k, (long long)t->rows,
                       (long long)t->cols);
    if (t->cols > kMaxIndex && t->rows > 1 && t->stride != t->cols)
        return gs_fail(ctx, GS_ERR_OVERFLOW, "%s %d: strided rows of %lld values", what, k, (long long)t->cols);
    if (written && t->rows > 1 && t->stride < t->cols)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d: written rows overlap (stride %lld < cols %lld)", what, k,
                       (long long)t->stride, (long long)t->cols);
    if (!t->data || (uintptr_t)t->data % type_size(t->type))
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d: pointer NULL or not aligned to its element", what, k);
    return GS_OK;
}

gs_status check_index(gs_ctx* ctx, const void* idx, int32_t idx_type, int64_t n, int64_t rows, int64_t cols)
{
    if (idx_type != GS_I32 && idx_type != GS_I64)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "index type %d", idx_type);
    if (n < 0) return gs_fail(ctx, GS_ERR_INVALID_ARG, "negative index count");
    if (n > kMaxIndex || rows > kMaxIndex || cols > kMaxIndex)
        return gs_fail(ctx, GS_ERR_OVERFLOW, "%lld indices into %lld x %lld", (long long)n, (long long)rows,
                       (long long)cols);
    if (n > 0 && (!idx || (uintptr_t)idx % (idx_type == GS_I32 ? 4 : 8)))
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "index pointer NULL or not aligned");
    return GS_OK;
}

gs_status check_sizes(gs_ctx* ctx, const gs_tensor* a, const gs_tensor* b, const char* what, int32_t k)
{
    if (a->rows != b->rows || a->cols != b->cols)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d: %lld x %lld, expected %lld x %lld", what, k,
                       (long long)b->rows, (long long)b->cols, (long long)a->rows, (long long)a->cols);
    return GS_OK;
}

// a tensor that an update writes: of the parameter's sizes, contiguous, f32 unless it is a copy
gs_status check_contiguous(gs_ctx* ctx, const gs_tensor* t, const gs_tensor* param, bool f32, const char* what,
                           int32_t k)
{
    gs_status st = check_tensor(ctx, t, true, what, k);
    if (st == GS_OK) st = check_sizes(ctx, param, t, what, k);
    if (st != GS_OK) return st;
    if (f32 && t->type != GS_F32) return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d must be GS_F32", what, k);
    if (t->rows > 1 && t->cols > 0 && t->stride != t->cols)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d must be contiguous", what, k);
    return GS_OK;
}

// Runs a launcher with a list of workspaces of its own, released in stream
// order afterwards; no exception leaves.
template <typename F>
gs_status guarded(gs_ctx* ctx, F&& f)
{
    std::vector<GsAlloc> tmp;
    gs_status st;
    try {
        st = f(&tmp);
    } catch (...) {
        st = GS_ERR_OOM;
    }
    gs_free_all(ctx, &tmp);
    return st;
}

gs_status check_norm_args(gs_ctx* ctx, const gs_tensor* grads, int32_t n, double max_norm, const float* norm)
{
    if (n < 0 || (n > 0 && !grads)) return gs_fail(ctx, GS_ERR_INVALID_ARG, "gradient list");
    if (!(max_norm >= 0.0)) return gs_fail(ctx, GS_ERR_INVALID_ARG, "max_norm must be >= 0");
    if (!norm || (uintptr_t)norm % 4) return gs_fail(ctx, GS_ERR_INVALID_ARG, "norm pointer NULL or not aligned");
    int64_t total = 0;
    for (int32_t k = 0; k < n; ++k) {
        const gs_status st = check_tensor(ctx, grads + k, false, "gradient", k);
        if (st != GS_OK) return st;
        total += grads[k].rows * grads[k].cols;
        if (total > (1ll << 42)) return gs_fail(ctx, GS_ERR_OVERFLOW, "more than 2^42 values");
    }
    return GS_OK;
}

// A tensor of a layer whose values have the type `type`, or GS_F32 where
// `wide` allows it: rows x cols of a call.  NULL: not there.
gs_status check_part(gs_ctx* ctx, const gs_tensor* t, bool written, int type, bool wide, int64_t rows, int64_t cols,
                     const char* what)
{
    if (!t) return GS_OK;
    const gs_status st = check_tensor(ctx, t, written, what);
    if (st != GS_OK) return st;
    if (t->type != type && !(wide && t->type == GS_F32))
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s: element type %d with a layer of type %d", what, t->type, type);
    if (t->rows != rows || t->cols != cols)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s is %lld x %lld, expected %lld x %lld", what, (long long)t->rows,
                       (long long)t->cols, (long long)rows, (long long)cols);
    return GS_OK;
}

// What every layer call checks: x (n x in), w (outs x in, or 2 outs x in when
// gated), the activation and the n x outs tensor y (out or dout).
gs_status check_layer(gs_ctx* ctx, const gs_tensor* x, const gs_tensor* w, int32_t act, const gs_tensor* y,
                      bool written, bool gated, const char* what)
{
    gs_status st = check_tensor(ctx, x, false, "x");
    if (st == GS_OK) st = check_tensor(ctx, w, false, "w");
    if (st == GS_OK) st = check_tensor(ctx, y, written, what);
    if (st != GS_OK) return st;
    if (act < GS_ACT_NONE || act > GS_ACT_SIGMOID) return gs_fail(ctx, GS_ERR_INVALID_ARG, "activation %d", act);
    if (x->rows > kMaxIndex || x->cols > kMaxIndex || w->rows > kMaxIndex)
        return gs_fail(ctx, GS_ERR_OVERFLOW, "a layer of %lld rows from %lld to %lld columns", (long long)x->rows,
                       (long long)x->cols, (long long)w->rows);
    if (gated && w->rows % 2) return gs_fail(ctx, GS_ERR_INVALID_ARG, "a gated layer's w has gate and up rows");
    st = check_part(ctx, w, false, x->type, false, w->rows, x->cols, "w");
    if (st == GS_OK) st = check_part(ctx, y, written, x->type, true, x->rows, w->rows / (gated ? 2 : 1), what);
    return st;
}

gs_status check_linear_bwd(gs_ctx* ctx, const gs_tensor* x, const gs_tensor* w, const gs_tensor* pre, int32_t act,
                           const gs_tensor* dout, const gs_tensor* dx, const gs_tensor* dw, const gs_tensor* dbias,
                           bool gated)
{
    gs_status st = check_layer(ctx, x, w, act, dout, false, gated, "dout");
    if (st != GS_OK) return st;
    if (!pre && (gated || act != GS_ACT_NONE)) return gs_fail(ctx, GS_ERR_INVALID_ARG, "pre is NULL");
    if (gated || act != GS_ACT_NONE) st = check_part(ctx, pre, false, x->type, false, x->rows, w->rows, "pre");
    if (st == GS_OK) st = check_part(ctx, dx, true, x->type, false, x->rows, x->cols, "dx");
    if (st == GS_OK) st = check_part(ctx, dw, true, x->type, true, w->rows, x->cols, "dw");
    if (st == GS_OK) st = check_part(ctx, dbias, true, x->type, true, 1, w->rows, "dbias");
    return st;
}

}  // namespace

extern "C" {

gs_status gs_embed_fwd(gs_ctx* ctx, const gs_tensor* table, const void* idx, int32_t idx_type, int64_t n, float scale,
                       const gs_tensor* out)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    gs_status st = check_tensor(ctx, table, false, "table");
    if (st == GS_OK) st = check_tensor(ctx, out, true, "out");
    if (st == GS_OK) st = check_index(ctx, idx, idx_type, n, table->rows, table->cols);
    if (st != GS_OK) return st;
    if (out->rows != n || out->cols != table->cols)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "out is %lld x %lld, expected %lld x %lld", (long long)out->rows,
                       (long long)out->cols, (long long)n, (long long)table->cols);
    return guarded(ctx, [&](std::vector<GsAlloc>*) { return launch_embed_fwd(ctx, table, idx, idx_type, n, scale, out); });
}

gs_status gs_embed_bwd(gs_ctx* ctx, const void* idx, int32_t idx_type, int64_t n, const gs_tensor* dout, float scale,
                       int64_t padding, int32_t accumulate, const gs_tensor* dtable)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    gs_status st = check_tensor(ctx, dout, false, "dout");
    if (st == GS_OK) st = check_tensor(ctx, dtable, true, "dtable");
    if (st == GS_OK) st = check_index(ctx, idx, idx_type, n, dtable->rows, dtable->cols);
    if (st != GS_OK) return st;
    if (dout->rows != n || dout->cols != dtable->cols)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "dout is %lld x %lld, expected %lld x %lld", (long long)dout->rows,
                       (long long)dout->cols, (long long)n, (long long)dtable->cols);
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_embed_bwd(ctx, idx, idx_type, n, dout, scale, padding, accumulate != 0, dtable, tmp);
    });
}

gs_status gs_grad_norm(gs_ctx* ctx, const gs_tensor* grads, int32_t n_tensors, double max_norm, float* norm)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    const gs_status st = check_norm_args(ctx, grads, n_tensors, max_norm, norm);
    if (st != GS_OK) return st;
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_grad_norm(ctx, grads, n_tensors, max_norm, norm, tmp);
    });
}

gs_status gs_clip_grads(gs_ctx* ctx, const gs_tensor* grads, int32_t n_tensors, double max_norm, const gs_tensor* out,
                        float* norm)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    gs_status st = check_norm_args(ctx, grads, n_tensors, max_norm, norm);
    const gs_tensor* to = out ? out : grads;
    for (int32_t k = 0; st == GS_OK && k < n_tensors; ++k) {
        st = check_tensor(ctx, to + k, true, "clipped gradient", k);
        if (st == GS_OK) st = check_sizes(ctx, grads + k, to + k, "clipped gradient", k);
        if (st == GS_OK && to[k].type != grads[k].type)
            st = gs_fail(ctx, GS_ERR_INVALID_ARG, "clipped gradient %d: another type", k);
    }
    if (st != GS_OK) return st;
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_clip(ctx, grads, n_tensors, max_norm, to, norm, tmp);
    });
}

gs_status gs_adam_tensors(gs_ctx* ctx, const gs_tensor* params, const gs_tensor* m, const gs_tensor* v,
                          const gs_tensor* grads, const gs_tensor* copies, int32_t n_tensors,
                          const gs_adam_opts* opts, const float* norm)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    if (n_tensors < 0 || (n_tensors > 0 && (!params || !m || !v || !grads)) || !opts)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "gs_adam_tensors arguments");
    if (opts->step < 1 || !(opts->beta1 >= 0.0 && opts->beta1 < 1.0) || !(opts->beta2 >= 0.0 && opts->beta2 < 1.0) ||
        !(opts->eps >= 0.0) || !std::isfinite(opts->eps) || !std::isfinite(opts->lr) ||
        !std::isfinite(opts->weight_decay))
        return gs_fail(ctx, GS_ERR_INVALID_ARG,
                       "Adam options: step >= 1, 0 <= betas < 1, eps >= 0, lr and weight decay finite");
    if (norm && (uintptr_t)norm % 4) return gs_fail(ctx, GS_ERR_INVALID_ARG, "norm pointer not aligned");
    int64_t total = 0;
    for (int32_t k = 0; k < n_tensors; ++k) {
        const gs_tensor* own[4] = {params + k, m + k, v + k, copies && copies[k].data ? copies + k : nullptr};
        const char* name[4] = {"parameter", "first moment", "second moment", "copy"};
        for (int q = 0; q < 4; ++q) {
            if (!own[q]) continue;
            const gs_status st = check_contiguous(ctx, own[q], params + k, q < 3, name[q], k);
            if (st != GS_OK) return st;
        }
        gs_status st = check_tensor(ctx, grads + k, false, "gradient", k);
        if (st == GS_OK) st = check_sizes(ctx, params + k, grads + k, "gradient", k);
        if (st != GS_OK) return st;
        total += params[k].rows * params[k].cols;
        if (total > (1ll << 42)) return gs_fail(ctx, GS_ERR_OVERFLOW, "more than 2^42 values");
    }
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_adam_list(ctx, params, m, v, grads, copies, n_tensors, opts, norm, tmp);
    });
}

gs_status gs_linear_fwd(gs_ctx* ctx, const gs_tensor* x, const gs_tensor* w, const gs_tensor* bias, int32_t act,
                        const gs_tensor* residual, const gs_tensor* pre, const gs_tensor* out)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    gs_status st = check_layer(ctx, x, w, act, out, true, false, "out");
    if (st == GS_OK) st = check_part(ctx, bias, false, x->type, true, 1, w->rows, "bias");
    if (st == GS_OK) st = check_part(ctx, residual, false, x->type, true, x->rows, w->rows, "residual");
    if (st == GS_OK) st = check_part(ctx, pre, true, x->type, false, x->rows, w->rows, "pre");
    if (st != GS_OK) return st;
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_linear_fwd(ctx, x, w, bias, act, residual, pre, out, false, tmp);
    });
}

gs_status gs_linear_bwd(gs_ctx* ctx, const gs_tensor* x, const gs_tensor* w, const gs_tensor* pre, int32_t act,
                        const gs_tensor* dout, int32_t accumulate, const gs_tensor* dx, const gs_tensor* dw,
                        const gs_tensor* dbias)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    const gs_status st = check_linear_bwd(ctx, x, w, pre, act, dout, dx, dw, dbias, false);
    if (st != GS_OK) return st;
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_linear_bwd(ctx, x, w, act == GS_ACT_NONE ? nullptr : pre, act, dout, accumulate != 0, dx, dw, dbias,
                                 false, tmp);
    });
}

gs_status gs_gated_fwd(gs_ctx* ctx, const gs_tensor* x, const gs_tensor* w, int32_t act, const gs_tensor* pre,
                       const gs_tensor* out)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    gs_status st = check_layer(ctx, x, w, act, out, true, true, "out");
    if (st == GS_OK) st = check_part(ctx, pre, true, x->type, false, x->rows, w->rows, "pre");
    if (st != GS_OK) return st;
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_linear_fwd(ctx, x, w, nullptr, act, nullptr, pre, out, true, tmp);
    });
}

gs_status gs_gated_bwd(gs_ctx* ctx, const gs_tensor* x, const gs_tensor* w, const gs_tensor* pre, int32_t act,
                       const gs_tensor* dout, int32_t accumulate, const gs_tensor* dx, const gs_tensor* dw)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    const gs_status st = check_linear_bwd(ctx, x, w, pre, act, dout, dx, dw, nullptr, true);
    if (st != GS_OK) return st;
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_linear_bwd(ctx, x, w, pre, act, dout, accumulate != 0, dx, dw, nullptr, true, tmp);
    });
}

gs_status gs_muon_tensors(gs_ctx* ctx, const gs_tensor* params, const gs_tensor* m, const gs_tensor* grads,
                          const gs_tensor* copies, int32_t n_tensors, const gs_muon_opts* opts, const float* norm)
{
    if (!ctx) return GS_ERR_INVALID_ARG;
    if (n_tensors < 0 || (n_tensors > 0 && (!params || !m || !grads)) || !opts)
        return gs_fail(ctx, GS_ERR_INVALID_ARG, "gs_muon_tensors arguments");
    if (opts->steps < 0 || opts->steps > 20 || !(opts->momentum >= 0.0 && opts->momentum < 1.0) ||
        !std::isfinite(opts->lr) || !std::isfinite(opts->weight_decay))
        return gs_fail(ctx, GS_ERR_INVALID_ARG,
                       "Muon options: 0 <= steps <= 20, 0 <= momentum < 1, lr and weight decay finite");
    if (norm && (uintptr_t)norm % 4) return gs_fail(ctx, GS_ERR_INVALID_ARG, "norm pointer not aligned");
    int64_t total = 0;
    for (int32_t k = 0; k < n_tensors; ++k) {
        const gs_tensor* own[3] = {params + k, m + k, copies && copies[k].data ? copies + k : nullptr};
        const char* name[3] = {"parameter", "momentum", "copy"};
        for (int q = 0; q < 3; ++q) {
            if (!own[q]) continue;
            gs_status st = check_contiguous(ctx, own[q], params + k, q < 2, name[q], k);
            if (st != GS_OK) return st;
        }
        gs_status st = check_tensor(ctx, grads + k, false, "gradient", k);
        if (st == GS_OK) st = check_sizes(ctx, params + k, grads + k, "gradient", k);
        if (st != GS_OK) return st;
        if (params[k].rows > (1 << 20) || params[k].cols > (1 << 20))
            return gs_fail(ctx, GS_ERR_OVERFLOW, "matrix %d: %lld x %lld", k, (long long)params[k].rows,
                           (long long)params[k].cols);
        total += params[k].rows * params[k].cols;
        if (total > (1ll << 42)) return gs_fail(ctx, GS_ERR_OVERFLOW, "more than 2^42 values");
    }
    return guarded(ctx, [&](std::vector<GsAlloc>* tmp) {
        return launch_muon_list(ctx, params, m, grads, copies, n_tensors, opts, norm, tmp);
    });
}

}  // extern "C"
