// tensors_api.cpp -- the C ABI of the table and tensor-list calls (declared in
// include/gs.h): argument checks, workspaces and launches.
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
            gs_status st = check_tensor(ctx, own[q], true, name[q], k);
            if (st == GS_OK) st = check_sizes(ctx, params + k, own[q], name[q], k);
            if (st != GS_OK) return st;
            if (q < 3 && own[q]->type != GS_F32)
                return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d must be GS_F32", name[q], k);
            if (own[q]->rows > 1 && own[q]->cols > 0 && own[q]->stride != own[q]->cols)
                return gs_fail(ctx, GS_ERR_INVALID_ARG, "%s %d must be contiguous", name[q], k);
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

}  // extern "C"
