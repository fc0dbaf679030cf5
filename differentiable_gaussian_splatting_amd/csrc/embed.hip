// embed.hip -- rows of a table by index, and the table's gradient.
//
//   forward   out[i, c] = scale table[idx[i], c]
//   backward  dtable[v, c] = scale sum over {i : idx[i] = v} of dout[i, c]
//
// The backward groups the positions i by index with a stable sort, so that
// each row's sum runs over its positions in ascending order and needs no
// atomics: the result does not depend on timing.
#include "gs_device.h"
#include "gs_internal.h"
#include "gs_tensor.h"

namespace {

using gst::narrow;
using gst::with_type;

// idx[i] as a row of the table, or rows (a value no row has) when it is
// outside [0, rows) or equal to skip
template <typename I>
__device__ __forceinline__ uint32_t row_of(const I* __restrict__ idx, int64_t i, uint32_t rows, int64_t skip)
{
    const int64_t v = (int64_t)idx[i];
    return v >= 0 && v < (int64_t)rows && v != skip ? (uint32_t)v : rows;
}

// one thread per value of out
template <typename T, typename O, typename I>
__global__ __launch_bounds__(256) void k_embed_fwd(const T* __restrict__ table, int64_t tstride, uint32_t rows,
                                                   const I* __restrict__ idx, int64_t n, uint32_t cols, float scale,
                                                   O* __restrict__ out, int64_t ostride)
{
    const int64_t total = n * cols, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; k < total; k += step) {
        const int64_t i = k / cols;
        const uint32_t c = (uint32_t)(k - i * cols);
        const uint32_t r = row_of(idx, i, rows, -1);
        out[i * ostride + c] = r < rows ? narrow<O>(scale * (float)table[r * tstride + c]) : (O)0.0f;
    }
}

template <typename I>
__global__ __launch_bounds__(256) void k_embed_keys(const I* __restrict__ idx, int64_t n, uint32_t rows, int64_t skip,
                                                    uint32_t* __restrict__ keys, uint32_t* __restrict__ pos)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    keys[i] = row_of(idx, i, rows, skip);
    pos[i] = (uint32_t)i;
}

// one thread per value of dtable: the sum over its row's positions
template <typename T, typename O>
__global__ __launch_bounds__(256) void k_embed_sum(const T* __restrict__ dout, int64_t dstride,
                                                   const uint64_t* __restrict__ first, const uint32_t* __restrict__ pos,
                                                   uint32_t rows, uint32_t cols, float scale, int accumulate,
                                                   O* __restrict__ dtable, int64_t ostride)
{
    const int64_t total = (int64_t)rows * cols, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; k < total; k += step) {
        const int64_t v = k / cols;
        const uint32_t c = (uint32_t)(k - v * cols);
        const uint64_t a = first[v], b = first[v + 1];
        O* o = dtable + v * ostride + c;
        if (a == b) {
            if (!accumulate) *o = (O)0.0f;
            continue;
        }
        float s = 0.0f;
        for (uint64_t j = a; j < b; ++j) s += (float)dout[(int64_t)pos[j] * dstride + c];
        *o = narrow<O>(accumulate ? (float)*o + scale * s : scale * s);
    }
}

unsigned flat_grid(int64_t total) { return (unsigned)std::min<int64_t>(std::max<int64_t>(ceil_div(total, 256), 1), 1 << 20); }

}  // namespace

gs_status launch_embed_fwd(gs_ctx* ctx, const gs_tensor* table, const void* idx, int idx_type, int64_t n, float scale,
                           const gs_tensor* out)
{
    if (n == 0 || table->cols == 0) return GS_OK;
    GsTimerScope ts(ctx, "embed_fwd");
    with_type(table->type, [&](auto t) {
        with_type(out->type, [&](auto o) {
            using T = decltype(t);
            using O = decltype(o);
            const dim3 grid(flat_grid(n * table->cols));
            if (idx_type == GS_I32)
                hipLaunchKernelGGL((k_embed_fwd<T, O, int32_t>), grid, dim3(256), 0, ctx->stream,
                                   (const T*)table->data, table->stride, (uint32_t)table->rows, (const int32_t*)idx, n,
                                   (uint32_t)table->cols, scale, (O*)out->data, out->stride);
            else
                hipLaunchKernelGGL((k_embed_fwd<T, O, int64_t>), grid, dim3(256), 0, ctx->stream,
                                   (const T*)table->data, table->stride, (uint32_t)table->rows, (const int64_t*)idx, n,
                                   (uint32_t)table->cols, scale, (O*)out->data, out->stride);
        });
    });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

gs_status launch_embed_bwd(gs_ctx* ctx, const void* idx, int idx_type, int64_t n, const gs_tensor* dout, float scale,
                           int64_t padding, int accumulate, const gs_tensor* dtable, std::vector<GsAlloc>* tmp)
{
    const int64_t rows = dtable->rows;
    if (rows == 0 || dtable->cols == 0) return GS_OK;
    const int64_t m = std::max<int64_t>(n, 1);
    uint32_t* k0 = (uint32_t*)gs_malloc(ctx, 4 * m, GS_MEM_SCRATCH, tmp);
    uint32_t* v0 = (uint32_t*)gs_malloc(ctx, 4 * m, GS_MEM_SCRATCH, tmp);
    uint32_t* k1 = (uint32_t*)gs_malloc(ctx, 4 * m, GS_MEM_SCRATCH, tmp);
    uint32_t* v1 = (uint32_t*)gs_malloc(ctx, 4 * m, GS_MEM_SCRATCH, tmp);
    uint32_t* scratch = (uint32_t*)gs_malloc(ctx, 4 * radix_scratch_words(m), GS_MEM_SCRATCH, tmp);
    uint64_t* first = (uint64_t*)gs_malloc(ctx, 8 * (rows + 2), GS_MEM_SCRATCH, tmp);
    if (!k0 || !v0 || !k1 || !v1 || !scratch || !first) return GS_ERR_OOM;
    if (n > 0) {
        GsTimerScope ts(ctx, "embed_bwd");
        const dim3 grid((unsigned)ceil_div(n, 256));
        if (idx_type == GS_I32)
            hipLaunchKernelGGL((k_embed_keys<int32_t>), grid, dim3(256), 0, ctx->stream, (const int32_t*)idx, n,
                               (uint32_t)rows, padding, k0, v0);
        else
            hipLaunchKernelGGL((k_embed_keys<int64_t>), grid, dim3(256), 0, ctx->stream, (const int64_t*)idx, n,
                               (uint32_t)rows, padding, k0, v0);
    }
    bool second = false;
    gs_status st = launch_radix_sort(ctx, k0, v0, k1, v1, n, bits_for(rows + 1), &second, nullptr, 0, nullptr, scratch);
    if (st == GS_OK) st = launch_seg_offsets(ctx, second ? k1 : k0, n, rows + 1, 0xFFFFFFFFu, first);
    if (st != GS_OK) return st;
    GsTimerScope ts(ctx, "embed_bwd");
    with_type(dout->type, [&](auto t) {
        with_type(dtable->type, [&](auto o) {
            using T = decltype(t);
            using O = decltype(o);
            hipLaunchKernelGGL((k_embed_sum<T, O>), dim3(flat_grid(rows * dtable->cols)), dim3(256), 0, ctx->stream,
                               (const T*)dout->data, dout->stride, first, second ? v1 : v0, (uint32_t)rows,
                               (uint32_t)dtable->cols, scale, accumulate, (O*)dtable->data, dtable->stride);
        });
    });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}
