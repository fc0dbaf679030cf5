// layers.hip -- linear and gated layers: which kernel a call takes, how its
// matrix products are cut into tiles and splits, and the gradient of the
// activation with the bias gradient's column sums.
//
//   linear: out = act(x w^T + bias) + residual
//           dz = dout act'(pre), dx = dz w, dw = dz^T x, dbias = sum over rows of dz
//   gated:  [g u] = x w^T, out = act(g) u
//           dg = dout u act'(g), du = dout act(g), then as above
//
// Forward: few rows (layer_few.hip), narrow rows (layer_narrow.h), else tiles
// (layer_mm.h).  Backward: narrow rows in one pass, else dz, then two products.
#include <algorithm>

#include "layer_narrow.h"

namespace {

using namespace gsm;

constexpr int kDzThreads = 256;

// dz, four columns of a row per thread: tx threads side by side, 256 / tx rows
// at once, a block walks `rows` rows.  dz is rounded to the layer's type, as
// the matrix instructions take it (a gradient that passes between layers of
// that type would be rounded the same way; a second part of each value would
// double both products); the column sums are of the f32 values, one partial row
// per block row, so they do not depend on timing.
//
// f16 holds 2^-24 to 65504 only, and dout act'(pre), or dout times the other
// half of a gated layer, may lie anywhere in f32's range.  So f16 values of dz
// are scaled by a power of two first, which the products' epilogues take back.
// The call's scale brings the largest finite |dz| to [2^14, 2^15).  It serves
// dw, which sums over the rows, and dx too if no row's largest is below 2^-14 of
// that: then the lost part of a value is at most 2^-11 of it or 2^-25 of its
// row's largest.  Otherwise dx has a dz of its own, scaled row by row, so that
// rows do not meet.  The largest values are found in a pass of their own
// (k_dz_max; 8191 x 2049 -> 4097: 57 us of 576).
struct DzJob {
    const void *pre, *dout;
    void* dz;            // null: not wanted
    void* dz_rows;       // f16: by the rows' scales where these differ too much; null: not wanted
    float* sums;         // [row blocks][n], null: none
    void* dbias;         // or, where one block holds all rows, the gradient itself
    float* row_max;      // f16: [m][chunks], the largest |dz| of `chunk` columns,
    float* all_max;      // and [2][max_blocks], the largest and the least of these but 0 that a block saw
    float* row_down;     // f16: [m], what takes a row's scale back,
    float* all_down;     // and the call's
    int32_t* by_rows;    // f16: 1 if dz_rows is written
    int32_t dbias_type, accumulate;
    int64_t m, n;        // n: columns of dout
    int64_t ldpre, lddout, lddz, rows, chunk;
    int32_t act, dout_type, tx, col_blocks, chunks, max_blocks;
};

constexpr int kMaxBlocks = 2048;   // of the pass for the largest values

// columns n to n + 3 of row m of dz; gated: of dg, and du
template <typename S, bool GATED>
__device__ __forceinline__ void dz_of(const DzJob& g, int64_t m, int64_t n, int valid, f32x4& dz, f32x4& du)
{
    const int type = sizeof(S) == 4 ? GS_F32 : -1;
    dz = load4<S>(g.dout, m * g.lddout + n, g.dout_type, valid);
    if constexpr (GATED) {
        const f32x4 z = load4<S>(g.pre, m * g.ldpre + n, type, valid);
        const f32x4 u = load4<S>(g.pre, m * g.ldpre + g.n + n, type, valid);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = act_both(z[j], g.act);
            du[j] = dz[j] * v.x;
            dz[j] = dz[j] * u[j] * v.y;
        }
    } else if (g.act != GS_ACT_NONE) {
        const f32x4 z = load4<S>(g.pre, m * g.ldpre + n, type, valid);
#pragma unroll
        for (int j = 0; j < 4; ++j) dz[j] *= act_both(z[j], g.act).y;
    }
}

// the largest of a and the least of b over the block
__device__ __forceinline__ float2 block_range(float a, float b, float2* part)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        a = fmaxf(a, __shfl_xor(a, d));
        b = fminf(b, __shfl_xor(b, d));
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kDzThreads / 64; ++w) {
        a = fmaxf(a, part[w].x);
        b = fminf(b, part[w].y);
    }
    return make_float2(a, b);
}

// the largest finite |dz| of each row, by chunks of its columns, and of each block
template <bool GATED>
__global__ __launch_bounds__(kDzThreads) void k_dz_max(const DzJob g)
{
    __shared__ float2 part[kDzThreads / 64];
    const int lane = threadIdx.x & 63, x = lane % g.tx, y = lane / g.tx, ny = 64 / g.tx;
    const int64_t groups = (g.m + ny - 1) / ny * g.chunks, stride = (int64_t)gridDim.x * (kDzThreads / 64);
    float all = 0.0f, least = INFINITY;
    for (int64_t t = (int64_t)blockIdx.x * (kDzThreads / 64) + (threadIdx.x >> 6); t < groups; t += stride) {
        const int64_t m = t / g.chunks * ny + y, c = t % g.chunks, end = min(g.n, (c + 1) * g.chunk);
        float most = 0.0f;
        auto take = [&](int64_t n, int valid) {
            f32x4 dz, du;
            dz_of<gst::f16, GATED>(g, m, n, valid, dz, du);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                most = larger(most, dz[j]);
                if constexpr (GATED) most = larger(most, du[j]);
            }
        };
        if (m < g.m) {
            int64_t n = c * g.chunk + x * 4;
#pragma unroll 2
            for (; n + 4 <= end; n += g.tx * 4) take(n, 4);
            if (n < end) take(n, (int)(end - n));
        }
        for (int d = 1; d < g.tx; d <<= 1) most = fmaxf(most, __shfl_xor(most, d));
        if (x == 0 && m < g.m) g.row_max[m * g.chunks + c] = most;
        all = fmaxf(all, most);
        if (most > 0.0f) least = fminf(least, most);
    }
    const float2 v = block_range(all, least, part);
    if (threadIdx.x == 0) {
        g.all_max[blockIdx.x] = v.x;
        g.all_max[gridDim.x + blockIdx.x] = v.y;
    }
}

template <typename S, bool GATED>
__global__ __launch_bounds__(kDzThreads) void k_dz(const DzJob g)
{
    constexpr bool kScaled = std::is_same<S, gst::f16>::value;
    __shared__ f32x4 part[kDzThreads];
    const int x = threadIdx.x % g.tx, y = threadIdx.x / g.tx, ny = kDzThreads / g.tx;
    const int type = sizeof(S) == 4 ? GS_F32 : -1;
    const int64_t cb = blockIdx.x % g.col_blocks, rb = blockIdx.x / g.col_blocks;
    const int64_t n = (cb * g.tx + x) * 4, end = min(g.m, (rb + 1) * g.rows);
    const int valid = (int)min((int64_t)4, g.n - n);
    float up = 1.0f;   // the call's scale
    bool by_rows = false;
    if constexpr (kScaled) {
        if (g.row_max) {
            float most = 0.0f, least = INFINITY;
            for (int b = threadIdx.x; b < g.max_blocks; b += kDzThreads) {
                most = fmaxf(most, g.all_max[b]);
                least = fminf(least, g.all_max[g.max_blocks + b]);
            }
            const float2 v = block_range(most, least, reinterpret_cast<float2*>(part));
            __syncthreads();   // part is free again
            const int e = scale_exponent(v.x);
            up = ldexpf(1.0f, e);
            by_rows = g.dz_rows && v.y * 16384.0f < v.x;
            if (blockIdx.x == 0 && threadIdx.x == 0) {
                *g.all_down = ldexpf(1.0f, -e);
                *g.by_rows = by_rows;
            }
        }
    }
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (valid > 0) {
        for (int64_t m = rb * g.rows + y; m < end; m += ny) {
            f32x4 dz, du;
            float most = 0.0f;
            if (kScaled && by_rows) most = g.row_max[m * g.chunks];
            dz_of<S, GATED>(g, m, n, valid, dz, du);
            if constexpr (kScaled) {
                float own = up;
                if (by_rows) {
                    for (int c = 1; c < g.chunks; ++c) most = fmaxf(most, g.row_max[m * g.chunks + c]);
                    own = ldexpf(1.0f, scale_exponent(most));
                    store4<S>(g.dz_rows, m * g.lddz + n, type, valid, dz * own);
                    if constexpr (GATED) store4<S>(g.dz_rows, m * g.lddz + g.n + n, type, valid, du * own);
                }
                if (g.row_down && cb == 0 && x == 0) g.row_down[m] = 1.0f / own;
            }
            if constexpr (GATED) {
                store4<S>(g.dz, m * g.lddz + g.n + n, type, valid, kScaled ? du * up : du);
                store4<S>(g.dz, m * g.lddz + n, type, valid, kScaled ? dz * up : dz);
            } else {
                if (g.dz) store4<S>(g.dz, m * g.lddz + n, type, valid, kScaled ? dz * up : dz);
                sum += dz;
            }
        }
    }
    if constexpr (!GATED) {
        if (!g.sums && !g.dbias) return;
        part[threadIdx.x] = sum;
        __syncthreads();
        if (y == 0 && valid > 0) {
            for (int q = 1; q < ny; ++q) sum += part[q * g.tx + x];
            if (g.dbias) {
                if (g.accumulate) sum += load4<S>(g.dbias, n, g.dbias_type, valid);
                store4<S>(g.dbias, n, g.dbias_type, valid, sum);
            } else {
                store4<float>(g.sums, rb * g.n + n, GS_F32, valid, sum);
            }
        }
    }
}

// Sums over `blocks` rows of f k + f values each, plus the old values when
// accumulate: the first f k of them to dw [f][k], the others to dbias (either
// null: not wanted).  64 columns a block, four quarters of the rows.
struct SumJob {
    const float* sums;
    void *dw, *dbias;
    int64_t blocks, f, k, lddw;
    int32_t dw_type, dbias_type, accumulate;
};

template <typename S>
__global__ __launch_bounds__(256) void k_sum_rows(const SumJob g)
{
    __shared__ float part[4][64];
    const int x = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t n = g.f * g.k + g.f;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < n; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + x;
        const bool weight = c < g.f * g.k, wanted = c < n && (weight ? g.dw : g.dbias);
        float s = 0.0f;
        if (wanted) {
#pragma unroll 8
            for (int64_t b = q; b < g.blocks; b += 4) s += g.sums[b * n + c];
        }
        part[q][x] = s;
        __syncthreads();
        if (q == 0 && wanted) {
            s = (part[0][x] + part[1][x]) + (part[2][x] + part[3][x]);
            const int type = weight ? g.dw_type : g.dbias_type;
            const int64_t at = weight ? c / g.k * g.lddw + c % g.k : c - g.f * g.k;
            void* out = weight ? g.dw : g.dbias;
            if (type == GS_F32) {
                float* o = (float*)out + at;
                *o = g.accumulate ? *o + s : s;
            } else {
                S* o = (S*)out + at;
                *o = gst::narrow<S>(g.accumulate ? (float)*o + s : s);
            }
        }
        __syncthreads();
    }
}

gs_status launch_sum_rows(gs_ctx* ctx, int type, const SumJob& g)
{
    GsTimerScope ts(ctx, "layer_sum");
    gst::with_type(type, [&](auto s) {
        hipLaunchKernelGGL((k_sum_rows<decltype(s)>), dim3((uint32_t)std::min<int64_t>(ceil_div(g.f * g.k + g.f, 64), 1 << 20)),
                           dim3(256), 0, ctx->stream, g);
    });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

// The tile of a product and the tiles that are split (layer_plan.h).  Returns the floats of its workspace.
int64_t plan(const gs_ctx* ctx, bool f32, LayerMm* g)
{
    const TilePlan p = plan_tiles(ctx->num_cu, f32, loads_direct(*g),
                                  ProductShape{g->m, g->e.n, g->k, g->a_col, g->b_col, g->gated});
    g->tile = p.tile;
    g->tm = p.tm;
    g->tn = p.tn;
    g->full = p.full;
    g->splits = p.splits;
    g->kper = p.kper;
    g->ws = nullptr;
    return p.floats;
}

gs_status launch_mm(gs_ctx* ctx, int type, const LayerMm& g)
{
    if (g.m == 0 || g.e.n == 0) return GS_OK;
    return type == GS_F32 ? launch_layer_mm_f32(ctx, g) :
           type == GS_F16 ? launch_layer_mm_f16(ctx, g) : launch_layer_mm_bf16(ctx, g);
}

gs_status launch_pair(gs_ctx* ctx, int type, const LayerMm& x, const LayerMm& w)
{
    return type == GS_F32 ? launch_layer_pair_f32(ctx, x, w) :
           type == GS_F16 ? launch_layer_pair_f16(ctx, x, w) : launch_layer_pair_bf16(ctx, x, w);
}

Operand operand(const void* p, int64_t ld, int64_t rows, int64_t gate = 0)
{
    return Operand{p, ld, rows, 1.0f, (int32_t)gate};
}

}  // namespace

static gs_status check_launch(gs_ctx* ctx)
{
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

static void launch_narrow(gs_ctx* ctx, int type, const LayerMm& g)
{
    GsTimerScope ts(ctx, "layer_narrow");
    if (type == GS_F32) launch_narrow_fwd_f32(ctx, g);
    else if (type == GS_F16) launch_narrow_fwd_f16(ctx, g);
    else launch_narrow_fwd_bf16(ctx, g);
}

static void launch_narrow(gs_ctx* ctx, int type, const NarrowBwd& g, int64_t blocks)
{
    GsTimerScope ts(ctx, "layer_narrow");
    if (type == GS_F32) launch_narrow_bwd_f32(ctx, g, blocks);
    else if (type == GS_F16) launch_narrow_bwd_f16(ctx, g, blocks);
    else launch_narrow_bwd_bf16(ctx, g, blocks);
}

gs_status launch_linear_fwd(gs_ctx* ctx, const gs_tensor* x, const gs_tensor* w, const gs_tensor* bias, int act,
                            const gs_tensor* residual, const gs_tensor* pre, const gs_tensor* out, bool gated,
                            std::vector<GsAlloc>* tmp)
{
    LayerMm g{};
    g.m = out->rows;
    g.k = x->cols;
    g.gated = gated;
    g.a = operand(x->data, x->stride, x->rows);
    g.b = operand(w->data, w->stride, w->rows, gated ? out->cols : 0);
    g.e.n = out->cols;
    g.e.act = act;
    if (bias) g.e.bias = bias->data, g.e.bias_type = (int8_t)bias->type;
    if (residual) g.e.res = residual->data, g.e.ldres = residual->stride, g.e.res_type = (int8_t)residual->type;
    if (pre) g.e.pre = pre->data, g.e.ldpre = pre->stride, g.e.pre_type = (int8_t)pre->type;
    g.e.out = out->data, g.e.ldout = out->stride, g.e.out_type = (int8_t)out->type;
    if (g.m == 0 || g.e.n == 0) return GS_OK;
    if (few_rows(g)) return launch_layer_few(ctx, x->type, g);
    if (narrow_fwd(x->type, g)) {
        launch_narrow(ctx, x->type, g);
        return check_launch(ctx);
    }
    const int64_t ws = plan(ctx, x->type == GS_F32, &g);
    if (ws && !(g.ws = (float*)gs_malloc(ctx, 4 * ws, GS_MEM_SCRATCH, tmp))) return GS_ERR_OOM;
    return launch_mm(ctx, x->type, g);
}

gs_status launch_linear_bwd(gs_ctx* ctx, const gs_tensor* x, const gs_tensor* w, const gs_tensor* pre, int act,
                            const gs_tensor* dout, int accumulate, const gs_tensor* dx, const gs_tensor* dw,
                            const gs_tensor* dbias, bool gated, std::vector<GsAlloc>* tmp)
{
    const int type = x->type;
    const int64_t size = type == GS_F32 ? 4 : 2, m = x->rows, k = x->cols, n = w->rows;
    if (!gated && m > 0 && n > 0 && k > 0 && narrow_bwd(n, k)) {
        const bool sums = dw || dbias;
        NarrowBwd z{};
        z.x = x->data, z.ldx = x->stride;
        z.w = w->data, z.ldw = w->stride;
        if (pre) z.pre = pre->data, z.ldpre = pre->stride;
        z.dout = dout->data, z.lddout = dout->stride, z.dout_type = dout->type;
        if (dx) z.dx = dx->data, z.lddx = dx->stride;
        z.m = m, z.f = (int32_t)n, z.k = (int32_t)k, z.act = act;
        const int64_t blocks = narrow_blocks(ctx, type, m, n, k);
        if (!sums && !dx) return GS_OK;
        if (sums && !(z.sums = (float*)gs_malloc(ctx, 4 * blocks * (n * k + n), GS_MEM_SCRATCH, tmp))) return GS_ERR_OOM;
        launch_narrow(ctx, type, z, blocks);
        gs_status st = check_launch(ctx);
        if (st != GS_OK || !sums) return st;
        return launch_sum_rows(ctx, type, SumJob{z.sums, dw ? dw->data : nullptr, dbias ? dbias->data : nullptr, blocks, n, k,
                                                 dw ? dw->stride : 0, dw ? dw->type : 0, dbias ? dbias->type : 0, accumulate});
    }
    // dz, the layer's dout itself where nothing changes it
    const bool own = m * n > 0 && (gated || act != GS_ACT_NONE || dout->type != type) && (dx || dw);
    const bool scaled = own && type == GS_F16;
    DzJob z{};
    int64_t row_blocks = 0;
    if (own || (dbias && m > 0)) {
        z.pre = pre ? pre->data : nullptr;
        z.ldpre = pre ? pre->stride : 0;
        z.dout = dout->data;
        z.lddout = dout->stride;
        z.dout_type = dout->type;
        z.act = act;
        z.m = m;
        z.n = dout->cols;
        const int64_t groups = ceil_div(z.n, 4);
        z.tx = 64;
        while (z.tx > 1 && z.tx / 2 >= groups) z.tx /= 2;
        z.col_blocks = (int32_t)ceil_div(groups, z.tx);
        const int ny = kDzThreads / z.tx;
        z.rows = ceil_div(std::max<int64_t>(ceil_div(m * z.col_blocks, 2048), m <= 64 ? 64 : 4 * ny), ny) * ny;
        row_blocks = ceil_div(m, z.rows);
        z.lddz = (n + 7) / 8 * 8;   // rows that start on 16 bytes
        if (own && !(z.dz = gs_malloc(ctx, m * z.lddz * size, GS_MEM_SCRATCH, tmp))) return GS_ERR_OOM;
        if (scaled) {
            // a wave takes whole rows, or where there are too few of them up to 64 pieces of one
            z.chunk = m >= 4096 ? ceil_div(z.n, 256) * 256 : std::max<int64_t>(1024, ceil_div(ceil_div(z.n, 64), 256) * 256);
            z.chunks = (int32_t)ceil_div(z.n, z.chunk);
            z.max_blocks = (int32_t)std::min<int64_t>(ceil_div(ceil_div(m, 64 / z.tx) * z.chunks, kDzThreads / 64), kMaxBlocks);
            if (!(z.row_max = (float*)gs_malloc(ctx, 4 * (m * z.chunks + m + 2 * kMaxBlocks + 2), GS_MEM_SCRATCH, tmp)))
                return GS_ERR_OOM;
            z.row_down = z.row_max + m * z.chunks;
            z.all_max = z.row_down + m;
            z.all_down = z.all_max + 2 * kMaxBlocks;
            z.by_rows = (int32_t*)(z.all_down + 1);
            if (dx && !(z.dz_rows = gs_malloc(ctx, m * z.lddz * size, GS_MEM_SCRATCH, tmp))) return GS_ERR_OOM;
        }
        if (dbias && row_blocks == 1) z.dbias = dbias->data, z.dbias_type = dbias->type, z.accumulate = accumulate;
        else if (dbias && !(z.sums = (float*)gs_malloc(ctx, 4 * row_blocks * n, GS_MEM_SCRATCH, tmp))) return GS_ERR_OOM;
    }
    const void* dz = own ? z.dz : dout->data;
    const int64_t lddz = own ? z.lddz : dout->stride;
    LayerMm gx{}, gw{};
    int64_t ws = 0, wsw = 0;
    if (dx && m * k > 0) {
        gx.m = m;
        gx.k = n;
        gx.b_col = true;
        gx.a = operand(dz, lddz, m);
        gx.b = operand(w->data, w->stride, k);
        gx.e.n = k;
        if (scaled) {
            gx.a_other = z.dz_rows;
            gx.other = z.by_rows;
            gx.e.down = z.row_down;
            gx.e.lddown = 1;
        }
        gx.e.out = dx->data, gx.e.ldout = dx->stride, gx.e.out_type = (int8_t)dx->type;
        ws = plan(ctx, type == GS_F32, &gx);
    }
    if (dw && n * k > 0) {
        gw.m = n;
        gw.k = m;
        gw.a_col = gw.b_col = true;
        gw.a = operand(dz, lddz, own ? lddz : n);   // own: the columns beside the last are there to be read
        gw.b = operand(x->data, x->stride, k);
        gw.e.n = k;
        if (scaled) gw.e.down = z.all_down;
        gw.e.out = dw->data, gw.e.ldout = dw->stride, gw.e.out_type = (int8_t)dw->type;
        if (accumulate) gw.e.res = dw->data, gw.e.ldres = dw->stride, gw.e.res_type = (int8_t)dw->type;
        wsw = plan(ctx, type == GS_F32, &gw);
    }
    // Small products share a launch: their tiles fill the card together, and a
    // launch costs the host 3 us (us apart / together: 148 rows of 234 -> 365
    // gated, 16-bit without f16's pass for the largest, 24.4 / 17.8, 2000 of 300 -> 300 f32 38.9 / 30.7; 43 of 4864 ->
    // 6912 bf16, where the products are long, 86 / 91).
    const bool pair = gx.m > 0 && gw.m > 0 && gx.tile == kSmall && gw.tile == kSmall &&
                      (double)m * (double)n * (double)k <= 5e8;
    float* sums = nullptr;   // of the splits; of both products, one after the other or side by side
    const int64_t floats = pair ? ws + wsw : std::max(ws, wsw);
    if (floats && !(sums = (float*)gs_malloc(ctx, 4 * floats, GS_MEM_SCRATCH, tmp))) return GS_ERR_OOM;
    gx.ws = sums;
    gw.ws = pair ? sums + ws : sums;

    if (z.m > 0 && z.n > 0) {
        GsTimerScope ts(ctx, "layer_dz");
        const dim3 grid((uint32_t)(row_blocks * z.col_blocks)), block(kDzThreads);
        if (scaled && gated) hipLaunchKernelGGL((k_dz_max<true>), dim3(z.max_blocks), block, 0, ctx->stream, z);
        else if (scaled) hipLaunchKernelGGL((k_dz_max<false>), dim3(z.max_blocks), block, 0, ctx->stream, z);
        auto go = [&](auto s) {
            typedef decltype(s) S;
            if (gated) hipLaunchKernelGGL((k_dz<S, true>), grid, block, 0, ctx->stream, z);
            else hipLaunchKernelGGL((k_dz<S, false>), grid, block, 0, ctx->stream, z);
        };
        gst::with_type(type, go);
        GS_HIP(ctx, hipGetLastError());
    }
    gs_status st = GS_OK;
    if (dbias && n > 0 && !z.dbias)
        st = launch_sum_rows(ctx, type, SumJob{z.sums, nullptr, dbias->data, row_blocks, n, 0, 0, 0, dbias->type, accumulate});
    if (st == GS_OK && pair) return launch_pair(ctx, type, gx, gw);
    if (st == GS_OK && gw.m > 0) st = launch_mm(ctx, type, gw);
    if (st == GS_OK && gx.m > 0) st = launch_mm(ctx, type, gx);
    return st;
}
