// layer_few.hip -- linear and gated layers of few rows (a step that adds one
// token per sequence, one view's embedding): the weights are read once and
// little else counts.
//
// A block owns 16 columns of out (and, gated, the 16 up rows that belong to
// them); its eight waves take eight ranges of k each, read their w rows
// straight from memory in the layout of the matrix instruction (a lane holds
// 16 bytes of one row: 16 rows x 64 bytes a load, eight neighbouring loads
// covering a 512-byte piece of each row), and add their sums up in LDS.  So
// every byte of w is loaded once by one lane, a wave has 8 KB under way, and no
// workspace or second launch is needed.  x comes out of the L2, once per block.
// f32 uses the f32 matrix instruction: the rate does not matter here.
//
// One row of 4096 x 4096 bf16: 9.0 us (3.7 TB/s); four rows of 2 x 11008 x 4096
// gated: 35 us (5.1 TB/s).  Sixteen waves a block take 9.6 us for the former;
// without the barrier before the products the compiler keeps two loads under
// way and the latter takes 40.
#include <algorithm>

#include "layer_mm.h"

namespace gsm {

namespace {

constexpr int kWaves = 8;

template <typename S, bool GATED, int MI>
__global__ __launch_bounds__(kWaves * 64) void k_few(const LayerMm g)
{
    constexpr int N = 16 / sizeof(S), kStep = 4 * N, G = GATED ? 2 : 1;   // values of a lane, and of a step of k
    constexpr int kUnroll = GATED || MI > 2 ? 4 : 8;
    __shared__ f32x4 part[kWaves][G][MI][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // ranges of whole pieces of kUnroll steps
    const int64_t piece = kStep * kUnroll, pieces = (g.k + piece - 1) / piece;
    const int64_t k0 = pieces * wave / kWaves * piece, k1 = min(pieces * (wave + 1) / kWaves * piece, g.k);
    const S* x[MI];
#pragma unroll
    for (int j = 0; j < MI; ++j)
        x[j] = (const S*)g.a.p + min((int64_t)(j * 16 + (lane & 15)), g.m - 1) * g.a.ld + (lane >> 4) * N;
    const int64_t up = GATED ? g.e.n * g.b.ld : 0;
    for (int64_t n0 = (int64_t)blockIdx.x * 16; n0 < g.e.n; n0 += (int64_t)gridDim.x * 16) {
        const S* w = (const S*)g.b.p + min(n0 + (lane & 15), g.e.n - 1) * g.b.ld + (lane >> 4) * N;
        f32x4 acc[G][MI];
#pragma unroll
        for (int q = 0; q < G; ++q)
#pragma unroll
            for (int j = 0; j < MI; ++j) acc[q][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        int64_t k = k0;
        for (; k + piece <= k1; k += piece) {
            gst::Pack<S, N> a[MI][kUnroll], b[G][kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
#pragma unroll
                for (int q = 0; q < G; ++q) b[q][i] = gst::load<S, N>(w + q * up + k + i * kStep);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
#pragma unroll
                for (int j = 0; j < MI; ++j) a[j][i] = gst::load<S, N>(x[j] + k + i * kStep);
            __builtin_amdgcn_sched_barrier(0);   // all loads under way before the first is waited for
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
#pragma unroll
                for (int q = 0; q < G; ++q)
#pragma unroll
                    for (int j = 0; j < MI; ++j) acc[q][j] = mfma16(b[q][i], a[j][i], acc[q][j]);
        }
        for (; k < k1; k += kStep) {
            const int64_t left = k1 - k - (lane >> 4) * N;
            gst::Pack<S, N> b[G];
#pragma unroll
            for (int q = 0; q < G; ++q) b[q] = upto<S, N>(w + q * up + k, left);
#pragma unroll
            for (int j = 0; j < MI; ++j) {
                const gst::Pack<S, N> a = upto<S, N>(x[j] + k, left);
#pragma unroll
                for (int q = 0; q < G; ++q) acc[q][j] = mfma16(b[q], a, acc[q][j]);
            }
        }
#pragma unroll
        for (int q = 0; q < G; ++q)
#pragma unroll
            for (int j = 0; j < MI; ++j) part[wave][q][j][lane] = acc[q][j];
        __syncthreads();
        // wave j adds the results of rows 16 j to 16 j + 15
        const int64_t n = n0 + (lane >> 4) * 4, m = wave * 16 + (lane & 15);
        if (wave < MI && m < g.m && n < g.e.n) {
            f32x4 sum[G];
#pragma unroll
            for (int q = 0; q < G; ++q) {
                sum[q] = part[0][q][wave][lane];
                for (int v = 1; v < kWaves; ++v) sum[q] += part[v][q][wave][lane];
            }
            if constexpr (GATED) epilogue_gated<S>(g.e, m, n, sum[0], sum[1]);
            else epilogue<S>(g.e, m, n, sum[0]);
        }
        __syncthreads();   // part is free again
    }
}

template <typename S, int MI>
void launch_few(gs_ctx* ctx, const LayerMm& g)
{
    const dim3 grid((uint32_t)std::min<int64_t>(ceil_div(g.e.n, 16), 1 << 20)), block(kWaves * 64);
    if (g.gated) hipLaunchKernelGGL((k_few<S, true, MI>), grid, block, 0, ctx->stream, g);
    else hipLaunchKernelGGL((k_few<S, false, MI>), grid, block, 0, ctx->stream, g);
}

}  // namespace

// Beyond 16 rows the tiles of k_layer_mm, which read x less often, become
// faster the larger w is.  us, here / tiles with splits, bf16: 32 rows of
// 1024 x 1024 6.5 / 10.4, of 4096 x 4096 15.2 / 17.3, of 11008 x 4096 38 / 26;
// 64 rows of 1024 x 1024 7.7 / 10.5, of 4096 x 4096 21.5 / 15.3.
bool few_rows(const LayerMm& g)
{
    const int64_t weights = g.e.n * (g.gated ? 2 : 1) * std::max<int64_t>(g.k, 1);
    return g.m <= 16 || (g.m <= 32 && weights <= 1 << 24) || (g.m <= 64 && weights <= 1 << 21);
}

gs_status launch_layer_few(gs_ctx* ctx, int type, const LayerMm& g)
{
    GsTimerScope ts(ctx, "layer_few");
    gst::with_type(type, [&](auto s) {
        typedef decltype(s) S;
        if (g.m <= 16) launch_few<S, 1>(ctx, g);
        else if (g.m <= 32) launch_few<S, 2>(ctx, g);
        else launch_few<S, 4>(ctx, g);
    });
    GS_HIP(ctx, hipGetLastError());
    return GS_OK;
}

}  // namespace gsm
